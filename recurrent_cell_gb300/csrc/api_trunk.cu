// api_trunk.cu -- the extern "C" entry points of the layer norm, the short
// convolution, the selective scan and gradient clipping (include/cfc.h).
//
// As in api.cu every argument is checked on the host before anything is enqueued;
// no allocation, no synchronisation, no host read of device data.
#include <algorithm>
#include <climits>
#include <initializer_list>
#include <new>

#include "cfc_internal.cuh"

namespace cfc {
namespace {

constexpr long long kMaxRows = 1ll << 30;
constexpr int kMaxSeqs = 1 << 20;
constexpr int kMaxChannels = 1 << 20;
constexpr int kMaxTensors = 65536;

bool aligned(std::initializer_list<const void*> ptrs, unsigned to) {
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) % to != 0) return false;
  return true;
}
bool missing(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!p) return true;
  return false;
}
int size_of(int math) { return math == CFC_MATH_BF16 ? 2 : 4; }
// a b, or the largest number where that is more (of a pool whose number of slots is the caller's).
long long times(long long a, long long b) {
  long long r;
  return __builtin_mul_overflow(a, b, &r) ? LLONG_MAX : r;
}
// What a call reads or writes: `rows` rows of `bytes` bytes, `pitch` apart (NULL: nothing).
struct Area {
  const void* at;
  long long rows, pitch, bytes;
};
Area dense(const void* p, long long bytes) { return Area{p, 1, 0, bytes}; }
Area spaced(const void* p, long long rows, long long ld, long long width, int math) {
  return Area{p, rows, ld * size_of(math), width * size_of(math)};
}
// Whether a dense area shares a byte with a row of another: with the first that ends behind its beginning.
bool meet(const Area& a, const Area& b) {
  if (!a.at || !b.at || a.rows < 1 || b.rows < 1 || a.bytes < 1 || b.bytes < 1) return false;
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.at), q = reinterpret_cast<uintptr_t>(b.at);
  const uintptr_t end = p + (uintptr_t)a.bytes, first = q + (uintptr_t)b.bytes;
  const uintptr_t k = p < first ? 0 : b.rows > 1 ? (p - first) / (uintptr_t)b.pitch + 1 : 1;
  return k < (uintptr_t)b.rows && q + k * (uintptr_t)b.pitch < end;
}
// Whether outputs (all dense) overlap neither inputs nor one another.
bool apart(std::initializer_list<Area> outs, std::initializer_list<Area> ins) {
  for (const Area* o = outs.begin(); o != outs.end(); ++o) {
    for (const Area* other = outs.begin(); other != o; ++other)
      if (meet(*o, *other)) return false;
    for (const Area& in : ins)
      if (meet(*o, in)) return false;
  }
  return true;
}
bool mode_ok(int math) { return math == CFC_MATH_FP32 || math == CFC_MATH_BF16; }
// Rows at least as far apart as they are wide, whole 16-byte vectors.
bool stride_ok(long long ld, long long width, int math) {
  return ld >= width && ld <= (1ll << 31) && ld % (16 / size_of(math)) == 0;
}
int done(cudaError_t e) { return e == cudaSuccess ? CFC_OK : CFC_ERR_LAUNCH; }
cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

// Sequences over rows: of a whole batch, or (tokens >= 0) of a step.
int check_sequences(long long rows, int n_seq, bool packed) {
  if (n_seq < 1 || n_seq > kMaxSeqs || rows < 0 || rows > kMaxRows) return CFC_ERR_SHAPE;
  if (!packed && rows % n_seq != 0) return CFC_ERR_SHAPE;
  return CFC_OK;
}
int check_step(int n_seq, int tokens, long long n_slots, const int* slots) {
  if (n_seq < 0 || n_seq > kMaxSeqs || tokens < 0 || n_slots < 0 || (long long)n_seq * tokens > kMaxRows) return CFC_ERR_SHAPE;
  return !slots && n_slots < n_seq ? CFC_ERR_SHAPE : CFC_OK;
}

// --- layer norm ----------------------------------------------------------------
int ln_check(long long rows, int d, int math) {
  if (!mode_ok(math)) return CFC_ERR_MODE;
  return rows < 0 || rows > (1ll << 40) || d < 1 || d > kMaxRmsWidth ? CFC_ERR_SHAPE : CFC_OK;
}

// --- short convolution -----------------------------------------------------------
int conv_check(int channels, int width, int math) {
  if (!mode_ok(math)) return CFC_ERR_MODE;
  return channels < 8 || channels > kMaxChannels || channels % 8 != 0 || width < 2 || width > kMaxConvWidth ? CFC_ERR_SHAPE
                                                                                                        : CFC_OK;
}
// Its outputs against its inputs and up to three more.
bool conv_apart(const ConvArgs& a, std::initializer_list<Area> outs, Area first = {}, Area second = {}, Area third = {}) {
  return apart(outs, {spaced(a.x, a.rows, a.ldx, a.d, a.math), dense(a.weight, 4ll * a.d * a.width), dense(a.bias, 4ll * a.d),
                      dense(a.off, 4ll * (a.n_seq + 1)), first, second, third});
}
// Blocks of a launch, one a tile of 16 rows and 128 vectors of 4 channels at most, and the states'.
bool conv_blocks_ok(long long rows, int n_seq, int channels) {
  return (rows / 16 + 1 + n_seq) * (channels / 4) / 128 < 0x7ffffff0ll;
}

// --- selective scan ----------------------------------------------------------------
int ssm_check(int channels, int groups, int n_states, int math) {
  if (!mode_ok(math)) return CFC_ERR_MODE;
  if (channels < 8 || channels > kMaxChannels || groups < 1 || channels % groups != 0 || channels / groups % 8 != 0)
    return CFC_ERR_SHAPE;
  if (n_states < 1 || n_states > kMaxSsmStates || (long long)groups * n_states > 65536) return CFC_ERR_SHAPE;
  return CFC_OK;
}
// What the three calls read.
struct SsmIn {
  SsmArgs a;
  int check_strides() const {
    const long long bc = (long long)a.groups * a.N;
    if (!stride_ok(a.ldx, a.d, a.math) || !stride_ok(a.ldd, a.d, a.math) || (a.z && !stride_ok(a.ldz, a.d, a.math)))
      return CFC_ERR_SHAPE;
    return a.ldb < bc || a.ldc < bc || a.ldb > (1ll << 31) || a.ldc > (1ll << 31) ? CFC_ERR_SHAPE : CFC_OK;
  }
  bool aligned_ok() const {
    return aligned({a.x, a.delta, a.z, a.init, a.ws}, 16) && aligned({a.B, a.C}, size_of(a.math)) &&
           aligned({a.A, a.D, a.bias, a.off}, 4);
  }
  bool null() const { return a.rows > 0 && missing({a.x, a.delta, a.A, a.B, a.C}); }
  bool apart(std::initializer_list<Area> outs, Area first = {}, Area second = {}) const {
    const long long bc = (long long)a.groups * a.N, d4 = 4ll * a.d;
    return cfc::apart(outs, {spaced(a.x, a.rows, a.ldx, a.d, a.math), spaced(a.delta, a.rows, a.ldd, a.d, a.math),
                             spaced(a.z, a.rows, a.ldz, a.d, a.math), spaced(a.B, a.rows, a.ldb, bc, a.math),
                             spaced(a.C, a.rows, a.ldc, bc, a.math), dense(a.A, d4 * a.N), dense(a.D, d4), dense(a.bias, d4),
                             dense(a.off, 4ll * (a.n_seq + 1)), dense(a.init, state_bytes()), first, second});
  }
  long long row_bytes() const { return a.rows * a.d * size_of(a.math); }
  long long state_bytes() const { return 4ll * a.n_seq * a.d * a.N; }
};
SsmIn ssm_in(const void* x, long long ldx, const void* delta, long long ldd, const float* A, const void* B, long long ldb,
             const void* C, long long ldc, const float* D, const void* z, long long ldz, const float* bias, const int* off,
             int n_seq, long long rows, int d, int groups, int N, int math, const float* init, void* ws) {
  SsmIn s{};
  SsmArgs& a = s.a;
  a.x = x; a.delta = delta; a.z = z; a.B = B; a.C = C;
  a.ldx = ldx; a.ldd = ldd; a.ldz = ldz; a.ldb = ldb; a.ldc = ldc;
  a.A = A; a.D = D; a.bias = bias; a.off = off; a.n_seq = n_seq; a.rows = rows;
  a.d = d; a.groups = groups; a.N = N; a.math = math; a.init = init; a.ws = static_cast<char*>(ws);
  return s;
}

}  // namespace
}  // namespace cfc

using namespace cfc;

extern "C" {

int cfc_layernorm_forward(const void* x, const void* residual, const float* weight, const float* bias, long long rows,
                          int d, float eps, int math, void* y, void* residual_out, float* mean, float* rstd, void* stream) {
  const int st = ln_check(rows, d, math);
  if (st != CFC_OK) return st;
  if (rows == 0) return CFC_OK;
  if (missing({x, weight, y})) return CFC_ERR_NULL;
  if (!aligned({x, residual, weight, bias, y, residual_out}, 16) || !aligned({mean, rstd}, 4)) return CFC_ERR_ALIGN;
  return done(launch_layernorm_forward(x, residual, weight, bias, rows, d, eps, math, y, residual_out, mean, rstd,
                                       as_stream(stream)));
}

size_t cfc_layernorm_workspace_bytes(long long rows, int d) {
  return ln_check(rows, d, CFC_MATH_FP32) == CFC_OK ? layernorm_workspace(rows, d) : 0;
}

int cfc_layernorm_backward(const void* s, const float* weight, const float* mean, const float* rstd, const void* grad_y,
                           const void* grad_residual_out, long long rows, int d, int math, void* grad_x,
                           float* grad_weight, float* grad_bias, void* workspace, size_t workspace_bytes, void* stream) {
  const int st = ln_check(rows, d, math);
  if (st != CFC_OK) return st;
  if (!grad_weight || (rows > 0 && missing({s, weight, mean, rstd, grad_y, grad_x}))) return CFC_ERR_NULL;
  if (!workspace || workspace_bytes < layernorm_workspace(rows, d)) return CFC_ERR_WORKSPACE;
  if (!aligned({s, weight, grad_y, grad_residual_out, grad_x, grad_weight, grad_bias, workspace}, 16) ||
      !aligned({mean, rstd}, 4))
    return CFC_ERR_ALIGN;
  return done(launch_layernorm_backward(s, weight, mean, rstd, grad_y, grad_residual_out, rows, d, math, grad_x, grad_weight,
                                        grad_bias, static_cast<float*>(workspace), as_stream(stream)));
}

int cfc_conv_forward(const void* x, long long x_stride, const float* weight, const float* bias, const int* seq_offsets,
                     int n_seq, long long rows, int channels, int width, int silu, int math, const void* initial_state,
                     void* y, void* final_state, void* stream) {
  int st = conv_check(channels, width, math);
  if (st == CFC_OK) st = check_sequences(rows, n_seq, seq_offsets != nullptr);
  if (st != CFC_OK) return st;
  if (!stride_ok(x_stride, channels, math) || !conv_blocks_ok(rows, n_seq, channels)) return CFC_ERR_SHAPE;
  if (!weight || (rows > 0 && missing({x, y}))) return CFC_ERR_NULL;
  if (!aligned({x, weight, initial_state, y, final_state}, 16) || !aligned({bias, seq_offsets}, 4)) return CFC_ERR_ALIGN;
  const ConvArgs a{x, x_stride, weight, bias, initial_state, seq_offsets, n_seq, rows, channels, width, silu != 0, math};
  const long long state = (long long)n_seq * (width - 1) * channels * size_of(math), out = rows * channels * size_of(math);
  if (!conv_apart(a, {dense(y, out), dense(final_state, state)}, dense(initial_state, state))) return CFC_ERR_OVERLAP;
  return done(launch_conv_forward(a, y, final_state, as_stream(stream)));
}

size_t cfc_conv_workspace_bytes(long long rows, int channels, int width, int math) {
  if (rows < 0 || rows > kMaxRows || conv_check(channels, width, math) != CFC_OK) return 0;
  return conv_workspace(rows, channels, width);
}

int cfc_conv_backward(const void* x, long long x_stride, const float* weight, const float* bias, const int* seq_offsets,
                      int n_seq, long long rows, int channels, int width, int silu, int math, const void* initial_state,
                      const void* grad_y, const void* grad_final_state, void* grad_x, float* grad_weight, float* grad_bias,
                      void* grad_initial_state, void* workspace, size_t workspace_bytes, void* stream) {
  int st = conv_check(channels, width, math);
  if (st == CFC_OK) st = check_sequences(rows, n_seq, seq_offsets != nullptr);
  if (st != CFC_OK) return st;
  if (!stride_ok(x_stride, channels, math) || !conv_blocks_ok(rows, n_seq, channels)) return CFC_ERR_SHAPE;
  if (missing({weight, grad_weight}) || (rows > 0 && missing({x, grad_y, grad_x}))) return CFC_ERR_NULL;
  if (!workspace || workspace_bytes < conv_workspace(rows, channels, width)) return CFC_ERR_WORKSPACE;
  if (!aligned({x, weight, initial_state, grad_y, grad_final_state, grad_x, grad_weight, grad_initial_state, workspace}, 16) ||
      !aligned({bias, seq_offsets, grad_bias}, 4))
    return CFC_ERR_ALIGN;
  const ConvArgs a{x, x_stride, weight, bias, initial_state, seq_offsets, n_seq, rows, channels, width, silu != 0, math};
  const long long state = (long long)n_seq * (width - 1) * channels * size_of(math), out = rows * channels * size_of(math);
  if (!conv_apart(a, {dense(grad_x, out), dense(grad_weight, 4ll * channels * width), dense(grad_bias, 4ll * channels),
                      dense(grad_initial_state, state), dense(workspace, conv_workspace(rows, channels, width))},
                  dense(initial_state, state), dense(grad_y, out), dense(grad_final_state, state)))
    return CFC_ERR_OVERLAP;
  return done(launch_conv_backward(a, grad_y, grad_final_state, grad_x, grad_weight, grad_bias, grad_initial_state,
                                   static_cast<float*>(workspace), as_stream(stream)));
}

int cfc_conv_step(const void* x, long long x_stride, const float* weight, const float* bias, int n_seq, int tokens,
                  int channels, int width, int silu, int math, void* state, long long n_slots, const int* slots, void* y,
                  void* stream) {
  int st = conv_check(channels, width, math);
  if (st == CFC_OK) st = check_step(n_seq, tokens, n_slots, slots);
  if (st != CFC_OK) return st;
  if (!stride_ok(x_stride, channels, math) || !conv_blocks_ok(0, n_seq, channels)) return CFC_ERR_SHAPE;
  if (n_seq == 0 || tokens == 0) return CFC_OK;
  if (missing({x, weight, y}) || (n_slots > 0 && !state)) return CFC_ERR_NULL;
  if (!aligned({x, weight, state, y}, 16) || !aligned({bias, slots}, 4)) return CFC_ERR_ALIGN;
  const long long rows = (long long)n_seq * tokens;
  const ConvArgs a{x, x_stride, weight, bias, nullptr, nullptr, n_seq, rows, channels, width, silu != 0, math};
  if (!conv_apart(a, {dense(y, rows * channels * size_of(math)),
                      dense(state, times(n_slots, (width - 1ll) * channels * size_of(math)))}, dense(slots, 4ll * n_seq)))
    return CFC_ERR_OVERLAP;
  return done(launch_conv_step(a, tokens, state, n_slots, slots, y, as_stream(stream)));
}

size_t cfc_ssm_workspace_bytes(long long rows, int n_seq, int channels, int groups, int n_states, int math, int save) {
  if (ssm_check(channels, groups, n_states, math) != CFC_OK || n_seq < 1 || n_seq > kMaxSeqs || rows < 0 || rows > kMaxRows)
    return 0;
  return ssm_workspace(rows, n_seq, channels, groups, n_states, save != 0);
}

int cfc_ssm_forward(const void* x, long long x_stride, const void* delta, long long delta_stride, const float* A,
                    const void* B, long long B_stride, const void* C, long long C_stride, const float* D, const void* z,
                    long long z_stride, const float* delta_bias, const int* seq_offsets, int n_seq, long long rows,
                    int channels, int groups, int n_states, int math, const float* initial_state, void* y,
                    float* final_state, int save, void* workspace, size_t workspace_bytes, void* stream) {
  int st = ssm_check(channels, groups, n_states, math);
  if (st == CFC_OK) st = check_sequences(rows, n_seq, seq_offsets != nullptr);
  if (st != CFC_OK) return st;
  const SsmIn in = ssm_in(x, x_stride, delta, delta_stride, A, B, B_stride, C, C_stride, D, z, z_stride, delta_bias,
                          seq_offsets, n_seq, rows, channels, groups, n_states, math, initial_state, workspace);
  if ((st = in.check_strides()) != CFC_OK) return st;
  if (in.null() || (rows > 0 && !y)) return CFC_ERR_NULL;
  const size_t need = ssm_workspace(rows, n_seq, channels, groups, n_states, save != 0);
  if (!workspace || workspace_bytes < need) return CFC_ERR_WORKSPACE;
  if (!in.aligned_ok() || !aligned({y, final_state}, 16)) return CFC_ERR_ALIGN;
  if (!in.apart({dense(y, in.row_bytes()), dense(final_state, in.state_bytes()), dense(workspace, need)})) return CFC_ERR_OVERLAP;
  return done(launch_ssm_forward(in.a, y, final_state, save != 0, as_stream(stream)));
}

int cfc_ssm_backward(const void* x, long long x_stride, const void* delta, long long delta_stride, const float* A,
                     const void* B, long long B_stride, const void* C, long long C_stride, const float* D, const void* z,
                     long long z_stride, const float* delta_bias, const int* seq_offsets, int n_seq, long long rows,
                     int channels, int groups, int n_states, int math, const float* initial_state, const void* grad_y,
                     const float* grad_final_state, void* grad_x, void* grad_delta, float* grad_A, void* grad_B,
                     void* grad_C, float* grad_D, void* grad_z, float* grad_delta_bias, float* grad_initial_state,
                     void* workspace, size_t workspace_bytes, void* stream) {
  int st = ssm_check(channels, groups, n_states, math);
  if (st == CFC_OK) st = check_sequences(rows, n_seq, seq_offsets != nullptr);
  if (st != CFC_OK) return st;
  const SsmIn in = ssm_in(x, x_stride, delta, delta_stride, A, B, B_stride, C, C_stride, D, z, z_stride, delta_bias,
                          seq_offsets, n_seq, rows, channels, groups, n_states, math, initial_state, workspace);
  if ((st = in.check_strides()) != CFC_OK) return st;
  if (in.null() || !grad_A || (rows > 0 && (missing({grad_y, grad_x, grad_delta, grad_B, grad_C}) || (z && !grad_z))))
    return CFC_ERR_NULL;
  const size_t need = ssm_workspace(rows, n_seq, channels, groups, n_states, 1);
  if (!workspace || workspace_bytes < need) return CFC_ERR_WORKSPACE;
  if (!in.aligned_ok() || !aligned({grad_y, grad_final_state, grad_x, grad_delta, grad_z, grad_initial_state}, 16) ||
      !aligned({grad_A, grad_B, grad_C, grad_D, grad_delta_bias}, 4))
    return CFC_ERR_ALIGN;
  const long long out = in.row_bytes(), bc = rows * groups * n_states * size_of(math), d4 = 4ll * channels;
  if (!in.apart({dense(grad_x, out), dense(grad_delta, out), dense(z ? grad_z : nullptr, out), dense(grad_B, bc), dense(grad_C, bc),
                 dense(grad_A, d4 * n_states), dense(grad_D, d4), dense(grad_delta_bias, d4),
                 dense(grad_initial_state, in.state_bytes()), dense(workspace, need)},
                dense(grad_y, out), dense(grad_final_state, in.state_bytes())))
    return CFC_ERR_OVERLAP;
  const SsmGrads r{grad_y, grad_final_state, grad_x, grad_delta, z ? grad_z : nullptr, grad_B, grad_C,
                   grad_A, grad_D, grad_delta_bias, grad_initial_state};
  return done(launch_ssm_backward(in.a, r, as_stream(stream)));
}

int cfc_ssm_step(const void* x, long long x_stride, const void* delta, long long delta_stride, const float* A,
                 const void* B, long long B_stride, const void* C, long long C_stride, const float* D, const void* z,
                 long long z_stride, const float* delta_bias, int n_seq, int tokens, int channels, int groups, int n_states,
                 int math, float* state, long long n_slots, const int* slots, void* y, void* stream) {
  int st = ssm_check(channels, groups, n_states, math);
  if (st == CFC_OK) st = check_step(n_seq, tokens, n_slots, slots);
  if (st != CFC_OK) return st;
  if ((long long)n_seq * (channels / 32 + 1) > 0x7fffffffll) return CFC_ERR_SHAPE;
  if (n_seq == 0 || tokens == 0) return CFC_OK;
  const SsmIn in = ssm_in(x, x_stride, delta, delta_stride, A, B, B_stride, C, C_stride, D, z, z_stride, delta_bias,
                          nullptr, n_seq, (long long)n_seq * tokens, channels, groups, n_states, math, nullptr, nullptr);
  if ((st = in.check_strides()) != CFC_OK) return st;
  if (in.null() || !y || (n_slots > 0 && !state)) return CFC_ERR_NULL;
  if (!in.aligned_ok() || !aligned({state, y}, 16) || !aligned({slots}, 4)) return CFC_ERR_ALIGN;
  if (!in.apart({dense(y, in.row_bytes()), dense(state, times(n_slots, 4ll * channels * n_states))}, dense(slots, 4ll * n_seq)))
    return CFC_ERR_OVERLAP;
  return done(launch_ssm_step(in.a, tokens, state, n_slots, slots, y, as_stream(stream)));
}

// --- gradient norm and clipping ----------------------------------------------------
size_t cfc_grad_clip_workspace_bytes(int count) {
  return count < 0 || count > kMaxTensors ? 0 : grad_workspace(count);
}

// Whether an output shares a byte with another tensor, its own gradient (in place) aside.
struct Span {
  uintptr_t at, end;
  bool out;
};
static int check_apart(const void* const* grads, void* const* out, const long long* n_values, const int* math, int count) {
  constexpr int kFew = 128;
  Span few[2 * kFew];
  Span* const spans = count <= kFew ? few : new (std::nothrow) Span[2 * (size_t)count];
  if (!spans) return CFC_ERR_LAUNCH;
  int n = 0;
  for (int i = 0; i < count; ++i) {
    if (n_values[i] == 0) continue;
    const uintptr_t bytes = (uintptr_t)n_values[i] * size_of(math[i]), p = reinterpret_cast<uintptr_t>(grads[i]),
                    q = reinterpret_cast<uintptr_t>(out[i]);
    spans[n++] = Span{q, q + bytes, true};
    if (p != q) spans[n++] = Span{p, p + bytes, false};
  }
  std::sort(spans, spans + n, [](const Span& a, const Span& b) { return a.at < b.at; });
  uintptr_t any = 0, written = 0;              // where those so far end
  bool meet = false;
  for (int i = 0; i < n; ++i) {
    meet |= spans[i].at < (spans[i].out ? any : written);
    any = std::max(any, spans[i].end);
    if (spans[i].out) written = std::max(written, spans[i].end);
  }
  if (spans != few) delete[] spans;
  return meet ? CFC_ERR_OVERLAP : CFC_OK;
}

static int grad_call(const void* const* grads, void* const* out, bool clip, const long long* n_values, const int* math,
                     int count, float max_norm, float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  if (count < 0 || count > kMaxTensors || !(max_norm >= 0.f)) return CFC_ERR_SHAPE;
  if (!norm || (count > 0 && (!grads || !n_values || !math || (clip && !out)))) return CFC_ERR_NULL;
  const long long need = grad_workspace(count);
  bool meets = meet(dense(norm, 4), dense(workspace, need));
  for (int i = 0; i < count; ++i) {
    if (!mode_ok(math[i])) return CFC_ERR_MODE;
    if (n_values[i] < 0 || n_values[i] > kMaxGradValues) return CFC_ERR_SHAPE;
    if (n_values[i] == 0) continue;
    if (!grads[i] || (clip && !out[i])) return CFC_ERR_NULL;
    if (!aligned({grads[i], clip ? out[i] : nullptr}, size_of(math[i]))) return CFC_ERR_ALIGN;
    // the sums, and in clipping the norm, are written while tensors are still to be read
    const long long bytes = n_values[i] * size_of(math[i]);
    for (const void* p : {grads[i], clip ? static_cast<const void*>(out[i]) : nullptr})
      meets |= meet(dense(workspace, need), dense(p, bytes)) || (clip && meet(dense(norm, 4), dense(p, bytes)));
  }
  if (!workspace || workspace_bytes < (size_t)need) return CFC_ERR_WORKSPACE;
  if (!aligned({workspace}, 16) || !aligned({norm}, 4)) return CFC_ERR_ALIGN;
  if (meets) return CFC_ERR_OVERLAP;
  if (const int st = clip ? check_apart(grads, out, n_values, math, count) : CFC_OK; st != CFC_OK) return st;
  return done(launch_grad_norm(grads, clip ? out : nullptr, n_values, math, count, max_norm, norm,
                               static_cast<double*>(workspace), as_stream(stream)));
}

int cfc_grad_norm(const void* const* grads, const long long* n_values, const int* math, int count, float* norm,
                  void* workspace, size_t workspace_bytes, void* stream) {
  return grad_call(grads, nullptr, false, n_values, math, count, 0.f, norm, workspace, workspace_bytes, stream);
}

int cfc_grad_clip(const void* const* grads, void* const* out, const long long* n_values, const int* math, int count,
                  float max_norm, float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  return grad_call(grads, out, true, n_values, math, count, max_norm, norm, workspace, workspace_bytes, stream);
}

}  // extern "C"
