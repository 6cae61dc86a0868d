// block_api.hip -- the C ABI of what stands around an attention block (declared
// in include/kda.h): the gated linear recurrence, the short convolution and the
// layer norm.  Host-side argument checks, workspace layout and the launches on
// the caller's stream.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "block_launch.h"
#include "kda.h"

namespace {

constexpr size_t ALIGN = 256;
constexpr int64_t I31 = (int64_t)1 << 31;
constexpr int32_t MAX_CHANNELS = 1 << 20;  // 32-bit offsets within a row, and grids over channels
constexpr int32_t MAX_WIDTH = 16384;       // channels of a row that a workgroup holds
constexpr int32_t MAX_TOKENS = INT32_MAX - 64;  // of a row of the batch: a tile may reach beyond its end

size_t align_up(size_t x) { return (x + ALIGN - 1) / ALIGN * ALIGN; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool aligned(std::initializer_list<const void*> ps, size_t a) {
    return std::all_of(ps.begin(), ps.end(), [a](const void* p) { return aligned(p, a); });
}
int status() { return hipGetLastError() == hipSuccess ? KDA_OK : KDA_ERR_LAUNCH; }
bool known_type(int32_t dtype) { return dtype == KDA_BF16 || dtype == KDA_FP32; }

// An array of a call, null or not.
struct Span {
    const void* p;
    size_t bytes;
};
bool meet(const Span& a, const Span& b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const uintptr_t i = (uintptr_t)a.p, j = (uintptr_t)b.p;
    return i < j + b.bytes && j < i + a.bytes;
}
// No output shares memory with an input or with another output.
bool apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        if (std::any_of(ins.begin(), ins.end(), [&](const Span& i) { return meet(*o, i); })) return false;
        if (std::any_of(o + 1, outs.end(), [&](const Span& q) { return meet(*o, q); })) return false;
    }
    return true;
}
// Each output is one of the inputs or shares no memory with them (for kernels in which
// whoever writes an element has read it).
bool in_place(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (const Span& o : outs)
        if (std::any_of(ins.begin(), ins.end(), [&](const Span& i) { return o.p != i.p && meet(o, i); })) return false;
    return true;
}
size_t token_bytes(int32_t dtype) { return dtype == KDA_FP32 ? 4 : 2; }

// Sizes of a batch of tokens; a status.
int check_batch(int32_t dtype, const int32_t* cu, int32_t num_seqs, int32_t B, int32_t T, int32_t C) {
    if (B < 1 || T < 0 || T > MAX_TOKENS || C < 1 || !known_type(dtype)) return KDA_ERR_INVALID_ARG;
    if (C % 8 || C > MAX_CHANNELS) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)B * T >= I31) return KDA_ERR_INVALID_ARG;
    if (cu && (B != 1 || num_seqs < 1 || !aligned(cu, 4))) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

bool valid_batch(int32_t B, int32_t T, int32_t C) {
    return B >= 1 && T >= 0 && T <= MAX_TOKENS && C >= 8 && C % 8 == 0 && C <= MAX_CHANNELS && (int64_t)B * T < I31;
}

int32_t scan_states(int32_t T) { return (int32_t)(((int64_t)T + kda::GS_STATES - 1) / kda::GS_STATES); }
int32_t scan_tiles(int32_t T) { return (int32_t)(((int64_t)T + kda::GS_TILE - 1) / kda::GS_TILE); }

// Tiles of all rows, of 64 channels and more, are counted in 32 bits (their tickets).
bool countable_tiles(int32_t B, int32_t T, int32_t C) {
    return (int64_t)B * scan_tiles(T) * ((C + 63) / 64) < I31;
}

// Workspace of the recurrence: the counters and words of the tiles (none where a row is one
// tile), a packed batch's marks and sequences, and for the gradients the tiles' sums.
struct ScanSpace {
    size_t tickets, words, marks, seq, part, total;
};

ScanSpace scan_space(int32_t B, int32_t T, int32_t C, bool packed, bool backward) {
    const size_t groups = packed ? ((size_t)T + 15) / 16 : 0;
    const bool one = T == 0 || (backward ? T <= kda::GS_TILE : !packed && T <= kda::GS_ONE_TILE);
    const int64_t counters = (int64_t)B * ((C + 63) / 64);
    ScanSpace s{};
    s.tickets = 0;
    s.words = one ? 0 : align_up((size_t)counters * kda::GS_TICKET_BYTES);
    s.marks = s.words + (one ? 0 : align_up((size_t)B * scan_tiles(T) * C * sizeof(uint64_t)));
    s.seq = s.marks + align_up(groups * sizeof(uint2));
    s.part = s.seq + align_up(groups * 16 * sizeof(int32_t));
    s.total = s.part + (backward ? align_up((size_t)B * scan_tiles(T) * 2 * C * sizeof(float)) : 0);
    return s;
}

int check_scan(const void* x, const void* g, const void* gate, const float* A_log, const float* dt_bias,
               const float* initial_state, const int32_t* cu, int32_t num_seqs, int32_t dtype, int32_t B, int32_t T,
               int32_t C) {
    const int st = check_batch(dtype, cu, num_seqs, B, T, C);
    if (st != KDA_OK) return st;
    if (!countable_tiles(B, T, C)) return KDA_ERR_INVALID_ARG;
    if (!A_log || !dt_bias || (T > 0 && (!x || !g || !gate))) return KDA_ERR_INVALID_ARG;
    if (!aligned({x, g, gate, initial_state}, 16) || !aligned({A_log, dt_bias}, 4)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

int check_workspace(const void* ws, size_t bytes, size_t need) {
    return !need || (ws && aligned(ws, ALIGN) && bytes >= need) ? KDA_OK : KDA_ERR_WORKSPACE;
}

kda::ScanArgs scan_args(const void* x, const void* g, const void* gate, const float* A_log, const float* dt_bias,
                        const float* initial_state, const int32_t* cu, int32_t num_seqs, int32_t B, int32_t T,
                        int32_t C, const ScanSpace& sp, void* workspace) {
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    kda::ScanArgs a{};
    a.x = x;
    a.g = g;
    a.gate = gate;
    a.A_log = A_log;
    a.dt_bias = dt_bias;
    a.h0 = initial_state;
    a.cu = cu;
    a.B = B;
    a.T = T;
    a.C = C;
    a.N = cu ? num_seqs : B;
    a.n_states = scan_states(T);
    a.tickets = reinterpret_cast<uint32_t*>(ws + sp.tickets);
    a.words = reinterpret_cast<uint64_t*>(ws + sp.words);
    a.marks = reinterpret_cast<uint2*>(ws + sp.marks);
    a.seq = reinterpret_cast<int32_t*>(ws + sp.seq);
    a.part = reinterpret_cast<float*>(ws + sp.part);
    return a;
}

int check_conv(const void* x, const float* weight, const float* bias, int32_t activation, const void* initial_state,
               const int32_t* cu, int32_t num_seqs, int32_t dtype, int32_t B, int32_t T, int32_t C, int32_t W) {
    const int st = check_batch(dtype, cu, num_seqs, B, T, C);
    if (st != KDA_OK) return st;
    if (W < 2 || W > 4) return KDA_ERR_UNSUPPORTED;
    if (activation != KDA_CONV_NONE && activation != KDA_CONV_SILU) return KDA_ERR_INVALID_ARG;
    if (!weight || (T > 0 && !x)) return KDA_ERR_INVALID_ARG;
    if (kda::short_conv_workgroups(B, T, C, cu ? num_seqs : B) >= I31) return KDA_ERR_INVALID_ARG;
    if (!aligned({x, initial_state}, 16) || !aligned({weight, bias}, 4)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

kda::ConvArgs conv_args(const void* x, const float* weight, const float* bias, int32_t activation,
                        const void* initial_state, const int32_t* cu, int32_t num_seqs, int32_t B, int32_t T,
                        int32_t C) {
    kda::ConvArgs a{};
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.silu = activation == KDA_CONV_SILU;
    a.h0 = initial_state;
    a.cu = cu;
    a.B = B;
    a.T = T;
    a.C = C;
    a.N = cu ? num_seqs : B;
    return a;
}

int check_layer_norm(const float* weight, float eps, int32_t dtype, int64_t rows, int32_t D) {
    if (rows < 0 || rows >= I31 || D < 1 || !known_type(dtype)) return KDA_ERR_INVALID_ARG;
    if (D % 8 || D > MAX_WIDTH) return KDA_ERR_UNSUPPORTED;
    if (!(eps >= 0.f) || !std::isfinite(eps) || !weight || !aligned(weight, 4)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

}  // namespace

extern "C" {

int64_t gated_scan_states(int32_t B, int32_t T, int32_t C) {
    return valid_batch(B, T, C) && countable_tiles(B, T, C) ? (int64_t)B * scan_states(T) * C : -1;
}

size_t gated_scan_fwd_workspace_size(int32_t B, int32_t T, int32_t C, int32_t packed) {
    if (!valid_batch(B, T, C) || !countable_tiles(B, T, C) || (packed && B != 1)) return 0;
    return std::max(ALIGN, scan_space(B, T, C, packed != 0, false).total);
}

size_t gated_scan_bwd_workspace_size(int32_t B, int32_t T, int32_t C, int32_t packed) {
    if (!valid_batch(B, T, C) || !countable_tiles(B, T, C) || (packed && B != 1)) return 0;
    return std::max(ALIGN, scan_space(B, T, C, packed != 0, true).total);
}

int gated_scan_fwd(const void* x, const void* g, const void* input_gate, const float* A_log, const float* dt_bias,
                   const float* initial_state, float* final_state, const int32_t* cu_seqlens, int32_t num_seqs,
                   int32_t dtype, int32_t B, int32_t T, int32_t C, void* o, float* states, void* workspace,
                   size_t workspace_bytes, void* stream) {
    int st = check_scan(x, g, input_gate, A_log, dt_bias, initial_state, cu_seqlens, num_seqs, dtype, B, T, C);
    if (st != KDA_OK) return st;
    if ((T > 0 && !o) || !aligned({o, final_state, states}, 16)) return KDA_ERR_INVALID_ARG;
    const ScanSpace sp = scan_space(B, T, C, cu_seqlens != nullptr, false);
    st = check_workspace(workspace, workspace_bytes, sp.total);
    if (st != KDA_OK) return st;
    const size_t tokens = (size_t)B * T * C * token_bytes(dtype), row = (size_t)C * sizeof(float);
    const size_t N = cu_seqlens ? num_seqs : B;
    const Span so{o, tokens}, sf{final_state, N * row}, ss{states, (size_t)B * scan_states(T) * row};
    const Span sw{workspace, sp.total}, sx{x, tokens}, sg{g, tokens}, si{input_gate, tokens};
    const Span sA{A_log, row}, sb{dt_bias, row}, s0{initial_state, N * row};
    const Span sc{cu_seqlens, (N + 1) * sizeof(int32_t)};
    if (!in_place({so}, {sx, sg, si}) || !apart({so, sf, ss, sw}, {sA, sb, s0, sc}) ||
        !apart({sf, ss, sw}, {sx, sg, si}))
        return KDA_ERR_INVALID_ARG;
    kda::ScanArgs a =
        scan_args(x, g, input_gate, A_log, dt_bias, initial_state, cu_seqlens, num_seqs, B, T, C, sp, workspace);
    a.h_final = final_state;
    a.o = o;
    a.states = states;
    (void)hipGetLastError();  // clear a stale error from unrelated work
    kda::launch_gated_scan_fwd(a, dtype == KDA_FP32, static_cast<hipStream_t>(stream));
    return status();
}

int gated_scan_bwd(const void* x, const void* g, const void* input_gate, const float* A_log, const float* dt_bias,
                   const float* initial_state, const int32_t* cu_seqlens, int32_t num_seqs, int32_t dtype, int32_t B,
                   int32_t T, int32_t C, const void* d_o, const float* d_final, const float* states, void* dx,
                   void* dg, void* dinput_gate, float* dA_log, float* ddt_bias, float* dh0, void* workspace,
                   size_t workspace_bytes, void* stream) {
    int st = check_scan(x, g, input_gate, A_log, dt_bias, initial_state, cu_seqlens, num_seqs, dtype, B, T, C);
    if (st != KDA_OK) return st;
    if (T > 0 && (!d_o || !states || !dx || !dg || !dinput_gate)) return KDA_ERR_INVALID_ARG;
    if (!dA_log || !ddt_bias || !aligned({dA_log, ddt_bias}, 4)) return KDA_ERR_INVALID_ARG;
    if (!aligned({d_o, d_final, states, dx, dg, dinput_gate, dh0}, 16)) return KDA_ERR_INVALID_ARG;
    const ScanSpace sp = scan_space(B, T, C, cu_seqlens != nullptr, true);
    st = check_workspace(workspace, workspace_bytes, sp.total);
    if (st != KDA_OK) return st;
    const size_t tokens = (size_t)B * T * C * token_bytes(dtype), row = (size_t)C * sizeof(float);
    const size_t N = cu_seqlens ? num_seqs : B;
    const Span gx{dx, tokens}, gg{dg, tokens}, gi{dinput_gate, tokens}, gA{dA_log, row}, gb{ddt_bias, row};
    const Span g0{dh0, N * row}, sw{workspace, sp.total};
    const Span sx{x, tokens}, sg{g, tokens}, si{input_gate, tokens}, sd{d_o, tokens};
    const Span sA{A_log, row}, sb{dt_bias, row}, s0{initial_state, N * row}, sf{d_final, N * row};
    const Span ss{states, (size_t)B * scan_states(T) * row}, sc{cu_seqlens, (N + 1) * sizeof(int32_t)};
    if (!in_place({gx, gg, gi}, {sx, sg, si, sd}) ||
        !apart({gx, gg, gi, gA, gb, g0, sw}, {sA, sb, s0, sf, ss, sc}) || !apart({gA, gb, g0, sw}, {sx, sg, si, sd}))
        return KDA_ERR_INVALID_ARG;
    kda::ScanArgs a =
        scan_args(x, g, input_gate, A_log, dt_bias, initial_state, cu_seqlens, num_seqs, B, T, C, sp, workspace);
    a.d_o = d_o;
    a.d_final = d_final;
    a.states = const_cast<float*>(states);  // (only read)
    a.dx = dx;
    a.dg = dg;
    a.dgate = dinput_gate;
    a.dA_log = dA_log;
    a.ddt_bias = ddt_bias;
    a.dh0 = dh0;
    (void)hipGetLastError();
    kda::launch_gated_scan_bwd(a, dtype == KDA_FP32, static_cast<hipStream_t>(stream));
    return status();
}

int gated_scan_decode(const void* x, const void* g, const void* input_gate, const float* A_log, const float* dt_bias,
                      const float* state_in, float* state_out, int32_t dtype, int32_t N, int32_t C, void* o,
                      void* stream) {
    const int st = check_batch(dtype, nullptr, 0, N, 1, C);
    if (st != KDA_OK) return st;
    if (!x || !g || !input_gate || !A_log || !dt_bias || !state_out || !o) return KDA_ERR_INVALID_ARG;
    if (!aligned({x, g, input_gate, state_in, state_out, o}, 16) || !aligned({A_log, dt_bias}, 4))
        return KDA_ERR_INVALID_ARG;
    const size_t tokens = (size_t)N * C * token_bytes(dtype), states = (size_t)N * C * sizeof(float);
    const Span so{o, tokens}, sn{state_out, states}, s0{state_in, states};
    const Span sx{x, tokens}, sg{g, tokens}, si{input_gate, tokens};
    const Span sA{A_log, C * sizeof(float)}, sb{dt_bias, C * sizeof(float)};
    if (!in_place({so}, {sx, sg, si}) || !in_place({sn}, {s0}) || !apart({so, sn}, {sA, sb}) || !apart({so}, {s0}) ||
        !apart({sn}, {sx, sg, si}))
        return KDA_ERR_INVALID_ARG;
    kda::ScanDecodeArgs a{};
    a.x = x;
    a.g = g;
    a.gate = input_gate;
    a.A_log = A_log;
    a.dt_bias = dt_bias;
    a.state_in = state_in;
    a.state_out = state_out;
    a.o = o;
    a.N = N;
    a.C = C;
    (void)hipGetLastError();
    kda::launch_gated_scan_decode(a, dtype == KDA_FP32, static_cast<hipStream_t>(stream));
    return status();
}

int short_conv_fwd(const void* x, const float* weight, const float* bias, int32_t activation,
                   const void* initial_state, void* final_state, const int32_t* cu_seqlens, int32_t num_seqs,
                   int32_t dtype, int32_t B, int32_t T, int32_t C, int32_t W, void* y, void* stream) {
    const int st = check_conv(x, weight, bias, activation, initial_state, cu_seqlens, num_seqs, dtype, B, T, C, W);
    if (st != KDA_OK) return st;
    if ((T > 0 && !y) || !aligned({y, final_state}, 16)) return KDA_ERR_INVALID_ARG;
    const size_t tokens = (size_t)B * T * C * token_bytes(dtype), row = (size_t)C * sizeof(float);
    const size_t N = cu_seqlens ? num_seqs : B, states = N * (W - 1) * C * token_bytes(dtype);
    if (!apart({{y, tokens}, {final_state, states}},
               {{x, tokens}, {initial_state, states}, {weight, W * row}, {bias, row},
                {cu_seqlens, (N + 1) * sizeof(int32_t)}}))
        return KDA_ERR_INVALID_ARG;
    kda::ConvArgs a = conv_args(x, weight, bias, activation, initial_state, cu_seqlens, num_seqs, B, T, C);
    a.h_final = final_state;
    a.y = y;
    (void)hipGetLastError();
    kda::launch_short_conv_fwd(a, W, dtype == KDA_FP32, static_cast<hipStream_t>(stream));
    return status();
}

size_t short_conv_bwd_workspace_size(int32_t dtype, int32_t B, int32_t T, int32_t C, int32_t W) {
    if (!valid_batch(B, T, C) || W < 2 || W > 4 || !known_type(dtype)) return 0;
    if (kda::short_conv_workgroups(B, T, C, B) >= I31) return 0;
    return std::max(
        ALIGN, align_up((size_t)kda::short_conv_groups(B, T, C, dtype == KDA_FP32) * (W + 1) * C * sizeof(float)));
}

int short_conv_bwd(const void* x, const float* weight, const float* bias, int32_t activation,
                   const void* initial_state, const int32_t* cu_seqlens, int32_t num_seqs, int32_t dtype, int32_t B,
                   int32_t T, int32_t C, int32_t W, const void* dy, const void* d_final, void* dx, float* dweight,
                   float* dbias, void* dh0, void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_conv(x, weight, bias, activation, initial_state, cu_seqlens, num_seqs, dtype, B, T, C, W);
    if (st != KDA_OK) return st;
    if (!dweight || (bias && !dbias) || (T > 0 && (!dy || !dx))) return KDA_ERR_INVALID_ARG;
    if (!aligned({dy, d_final, dx, dh0}, 16) || !aligned({dweight, dbias}, 4)) return KDA_ERR_INVALID_ARG;
    const size_t need = short_conv_bwd_workspace_size(dtype, B, T, C, W);
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != KDA_OK) return st;
    const size_t tokens = (size_t)B * T * C * token_bytes(dtype), row = (size_t)C * sizeof(float);
    const size_t N = cu_seqlens ? num_seqs : B, states = N * (W - 1) * C * token_bytes(dtype);
    if (!apart({{dx, tokens}, {dweight, W * row}, {dbias, row}, {dh0, states}, {workspace, need}},
               {{x, tokens}, {dy, tokens}, {initial_state, states}, {d_final, states}, {weight, W * row}, {bias, row},
                {cu_seqlens, (N + 1) * sizeof(int32_t)}}))
        return KDA_ERR_INVALID_ARG;
    kda::ConvArgs a = conv_args(x, weight, bias, activation, initial_state, cu_seqlens, num_seqs, B, T, C);
    a.dy = dy;
    a.d_final = d_final;
    a.dx = dx;
    a.dweight = dweight;
    a.dbias = dbias;
    a.dh0 = dh0;
    a.part = static_cast<float*>(workspace);
    (void)hipGetLastError();
    kda::launch_short_conv_bwd(a, W, dtype == KDA_FP32, static_cast<hipStream_t>(stream));
    return status();
}

int short_conv_decode(const void* x, const float* weight, const float* bias, int32_t activation,
                      const void* state_in, void* state_out, int32_t dtype, int32_t N, int32_t C, int32_t W, void* y,
                      void* stream) {
    const int st = check_conv(x, weight, bias, activation, state_in, nullptr, 0, dtype, N, 1, C, W);
    if (st != KDA_OK) return st;
    if (!state_in || !state_out || !y || !aligned({state_out, y}, 16)) return KDA_ERR_INVALID_ARG;
    const size_t tokens = (size_t)N * C * token_bytes(dtype), row = (size_t)C * sizeof(float);
    const Span sy{y, tokens}, sn{state_out, tokens * (W - 1)}, sx{x, tokens}, s0{state_in, tokens * (W - 1)};
    if (!in_place({sy}, {sx}) || !in_place({sn}, {s0}) || !apart({sy, sn}, {{weight, W * row}, {bias, row}}) ||
        !apart({sy}, {s0}) || !apart({sn}, {sx}))
        return KDA_ERR_INVALID_ARG;
    kda::ConvDecodeArgs a{};
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.state_in = state_in;
    a.state_out = state_out;
    a.y = y;
    a.N = N;
    a.C = C;
    a.silu = activation == KDA_CONV_SILU;
    (void)hipGetLastError();
    kda::launch_short_conv_decode(a, W, dtype == KDA_FP32, static_cast<hipStream_t>(stream));
    return status();
}

int layer_norm_fwd(const void* x, const void* residual, const float* weight, const float* bias, float eps,
                   int32_t dtype, int64_t rows, int32_t D, void* y, void* sum, void* stream) {
    const int st = check_layer_norm(weight, eps, dtype, rows, D);
    if (st != KDA_OK) return st;
    if (rows > 0 && (!x || !y || (residual && !sum))) return KDA_ERR_INVALID_ARG;
    if (!aligned({x, residual, y, sum}, 16) || !aligned(bias, 4)) return KDA_ERR_INVALID_ARG;
    if (rows == 0) return KDA_OK;
    const size_t tokens = (size_t)rows * D * token_bytes(dtype), row = (size_t)D * sizeof(float);
    const Span sy{y, tokens}, ss{residual ? sum : nullptr, tokens};
    if (!in_place({sy, ss}, {{x, tokens}, {residual, tokens}}) || !apart({sy, ss}, {{weight, row}, {bias, row}}))
        return KDA_ERR_INVALID_ARG;
    kda::LayerNormArgs a{};
    a.x = x;
    a.res = residual;
    a.weight = weight;
    a.bias = bias;
    a.eps = eps;
    a.D = D;
    a.rows = rows;
    a.y = y;
    a.sum = sum;
    (void)hipGetLastError();
    kda::launch_layer_norm_fwd(a, dtype == KDA_FP32, static_cast<hipStream_t>(stream));
    return status();
}

size_t layer_norm_bwd_workspace_size(int32_t dtype, int64_t rows, int32_t D) {
    if (rows < 0 || rows >= I31 || D < 8 || D % 8 || D > MAX_WIDTH || !known_type(dtype)) return 0;
    return align_up((size_t)kda::layer_norm_groups(rows, D, dtype == KDA_FP32) * 2 * D * sizeof(float));
}

int layer_norm_bwd(const void* sum, const float* weight, float eps, int32_t dtype, int64_t rows, int32_t D,
                   const void* dy, const void* dsum, void* dx, float* dweight, float* dbias, void* workspace,
                   size_t workspace_bytes, void* stream) {
    int st = check_layer_norm(weight, eps, dtype, rows, D);
    if (st != KDA_OK) return st;
    if (!dweight || (rows > 0 && (!sum || !dy || !dx))) return KDA_ERR_INVALID_ARG;
    if (!aligned({sum, dy, dsum, dx}, 16) || !aligned({dweight, dbias}, 4)) return KDA_ERR_INVALID_ARG;
    const size_t need = layer_norm_bwd_workspace_size(dtype, rows, D);
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != KDA_OK) return st;
    const size_t tokens = (size_t)rows * D * token_bytes(dtype), row = (size_t)D * sizeof(float);
    const Span gx{dx, tokens}, gw{dweight, row}, gb{dbias, row}, sw{workspace, need};
    const Span su{sum, tokens}, sd{dy, tokens}, ss{dsum, tokens};
    if (!in_place({gx}, {su, sd, ss}) || !apart({gx, gw, gb, sw}, {{weight, row}}) ||
        !apart({gw, gb, sw}, {su, sd, ss}))
        return KDA_ERR_INVALID_ARG;
    kda::LayerNormArgs a{};
    a.x = sum;
    a.weight = weight;
    a.eps = eps;
    a.D = D;
    a.rows = rows;
    a.dy = dy;
    a.dsum = dsum;
    a.dx = dx;
    a.dweight = dweight;
    a.dbias = dbias;
    a.part = static_cast<float*>(workspace);
    a.groups = kda::layer_norm_groups(rows, D, dtype == KDA_FP32);
    (void)hipGetLastError();
    kda::launch_layer_norm_bwd(a, dtype == KDA_FP32, static_cast<hipStream_t>(stream));
    return status();
}

}  // extern "C"
