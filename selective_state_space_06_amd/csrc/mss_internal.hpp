// mss_internal.hpp -- host-side launch descriptions passed from the validated C ABI
// (abi.hip) to the kernel launchers (scan_fwd.hip, state_update.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mss {

constexpr int kN = 16;      // d_state handled by the kernels
constexpr int kRows = 64;   // channels per wavefront (one lane per channel)
// Bytes of each row (per array) a fast-path tile covers: 64 for bf16 rows (half a 128-byte line:
// the LDS of two wavefronts per SIMD holds no more), a whole line for fp32 rows (one wavefront per
// SIMD leaves the LDS for it, and each line is then fetched once).
constexpr int fast_tile_bytes(bool bf16) { return bf16 ? 64 : 128; }

struct ScanLaunch {
    const void* u;
    const void* delta;
    const void* z;          // nullable
    const float* A;         // (Dn, N)
    const float* B;         // (Bt, N, L)
    const float* C;         // (Bt, N, L)
    const float* D;         // nullable
    const float* bias;      // nullable
    void* out;
    float* last_state;      // nullable
    const float* h0;        // nullable: starting state (Bt, Dn, N), zeros when null
    const int32_t* lens;    // nullable: per-batch sequence lengths (device), clamped to [0, L]
    float* saved;           // nullable: the state entering every 8-step tile, [ceil(L/8)][N][Bt*Dn]
    int64_t Bt, Dn, L;
    int N = 16;             // d_state: 16 (fast and general kernels), 32, 64 or 128 (general kernels)
    int softplus;
    bool bf16;              // storage type of u / delta / z / out
    bool vec_ok;            // rows of u / delta / z / out are 16-byte aligned
    // Optional timing events (all null or all valid): recorded on the stream before the first
    // kernel, before the main kernel and after it.
    hipEvent_t ev[3] = {nullptr, nullptr, nullptr};
};

// Records launch-timing event k of `a` on `stream` when timing is on.
inline void mark(const ScanLaunch& a, int k, hipStream_t stream) {
    if (a.ev[k]) (void)hipEventRecord(a.ev[k], stream);
}

struct DecodeLaunch {
    float* state;           // (Bt, Dn, N), in/out
    const void* x;
    const void* dt;
    const void* z;          // nullable
    const float* A;
    const float* B;         // (Bt, N)
    const float* C;         // (Bt, N)
    const float* D;         // nullable
    const float* bias;      // nullable
    void* out;
    int64_t Bt, Dn;
    int N;                  // d_state: 16, 32, 64 or 128
    bool bf16;
};

struct BwdLaunch {
    const void* u;
    const void* delta;
    const void* z;          // nullable
    const void* dout;
    const float* A;
    const float* B;
    const float* C;
    const float* D;         // nullable
    const float* bias;      // nullable
    void* du;
    void* ddelta;
    void* dz;               // nullable (also when z is null)
    float* dA;              // (Dn, N)
    float* dB;              // (Bt, N, L)
    float* dC;              // (Bt, N, L)
    float* dD;              // nullable
    float* dbias;           // nullable
    const float* h0;        // nullable: the forward's starting state (Bt, Dn, N)
    const int32_t* lens;    // nullable: per-batch sequence lengths (device)
    const float* dlast;     // nullable: dL/d last_state (Bt, Dn, N)
    float* dh0;             // nullable: dL/dh0 (Bt, Dn, N), written
    const float* saved;     // nullable: the forward's states entering every 8-step tile
                            // ([ceil(L/8)][N][Bt*Dn]); when given they replace the recomputation
    int64_t Bt, Dn, L;
    int softplus;
    bool bf16;
    bool vec_ok;            // rows of u / delta / z / dout / du / ddelta / dz and B / C 16-byte aligned
};

struct ConvLaunch {
    const void* x;          // (Bt, Dn, L)
    const float* w;         // (Dn, K)
    const float* bias;      // nullable
    const void* state_in;   // (Bt, Dn, K-1), nullable
    void* out;
    void* state_out;        // (Bt, Dn, K-1), nullable
    int64_t Dn, L, R;       // R = Bt * Dn
    int K;
    bool silu, bf16;
    bool vec_ok;            // rows of x / out span whole 16-byte vectors, 16-byte aligned
};

struct ConvUpdateLaunch {
    void* state;            // (Bt, Dn, K-1), in/out
    const void* x;          // (Bt, Dn)
    const float* w;
    const float* bias;
    void* out;
    int64_t Dn, R;
    int K;
    bool silu, bf16;
};

// Mamba-2 SSD layer (ssd_scan.hip): x, z, out (Bt, L, H, P); dt (Bt, L, H); B, C (Bt, L, G, N), all
// bf16; A, D, bias (H) fp32; last_state (Bt, H, P, N) fp32.  P = 64, N = 64 or 128.
struct SsdLaunch {
    const void* x;
    const void* dt;
    const float* A;
    const void* B;
    const void* C;
    const float* D;         // nullable
    const void* z;          // nullable
    const float* bias;      // nullable
    void* out;
    float* last_state;      // nullable
    int64_t Bt, L, H, P, G, N;
    int softplus;
};
// Segments per (batch, head) (segments_override > 0 replaces the count), the workspace they need,
// and the launch.
int plan_ssd_segments(const SsdLaunch& a, int num_cus, int segments_override);
size_t ssd_workspace_bytes(const SsdLaunch& a, int segments);
hipError_t launch_ssd_scan(const SsdLaunch& a, int segments, float* workspace, hipStream_t stream);

// How the forward scan is decomposed.  Generic path: `segments` workgroup-rows per channel
// group, each covering `seg_len` steps.  Fast path: `waves` wavefronts, each taking an equal
// contiguous range of the (channel group, tile) work; `segments` > 1 when some range ends
// inside a group (the aggregate kernel then has work).
struct ScanPlan {
    int segments;
    int64_t seg_len;
    int64_t waves;
    int64_t xcds;            // fast path: XCDs the wavefronts are dealt over
    bool fits = true;        // fast path: the (group, tile) count fits the kernels' 32-bit counts
    size_t workspace_bytes;  // carry workspace needed (0 when nothing is carried)
};

// Segment plan for a time tile of `tile` steps (segments are whole tiles).
ScanPlan plan_scan(const ScanLaunch& a, int num_cus, int tile, int segments_override);
// Generic path (any alignment): scan_fwd.hip.
hipError_t launch_scan_fwd(const ScanLaunch& a, const ScanPlan& plan, float* workspace,
                           hipStream_t stream);
int generic_tile();
size_t generic_workspace_bytes(const ScanLaunch& a, int segments);
// Fast path: scan_fast.hip.  `waves_override` > 0 replaces the automatic wavefront count.
ScanPlan plan_fast(const ScanLaunch& a, int num_cus, int64_t waves_override);
size_t fast_workspace_bytes(const ScanLaunch& a, const ScanPlan& plan);
hipError_t launch_scan_fast(const ScanLaunch& a, const ScanPlan& plan, float* workspace,
                            hipStream_t stream);
hipError_t launch_state_update(const DecodeLaunch& a, hipStream_t stream);
// Causal conv1d: conv1d.hip.
hipError_t launch_conv1d_fwd(const ConvLaunch& a, hipStream_t stream);
hipError_t launch_conv1d_update(const ConvUpdateLaunch& a, hipStream_t stream);
// Backward scan: scan_bwd.hip.
int plan_bwd_segments(const BwdLaunch& a, int num_cus, int segments_override);
size_t bwd_workspace_bytes(const BwdLaunch& a, int segments);
hipError_t launch_scan_bwd(const BwdLaunch& a, int segments, void* workspace, hipStream_t stream);

// Gated scan (gated_scan.hip): x, f, i, out and their gradients (Bt, Dn, L); rate (Dn); states (Bt, Dn).
constexpr int kGatedTile = 512;  // steps between two saved states

struct GatedLaunch {
    const void* x = nullptr;
    const void* f = nullptr;
    const void* i = nullptr;
    const float* rate = nullptr;
    const float* h0 = nullptr;       // nullable
    const int32_t* lens = nullptr;   // nullable
    void* out = nullptr;             // nullable when saved is given
    float* last_state = nullptr;     // nullable
    float* saved = nullptr;          // (Bt, Dn, ceil(L / 512)); the forward's is nullable
    // the backward's
    const void* dout = nullptr;
    const float* dlast = nullptr;    // nullable
    void* dx = nullptr;
    void* df = nullptr;
    void* di = nullptr;
    float* drate = nullptr;
    float* dh0 = nullptr;            // nullable
    float* scratch = nullptr;
    int64_t Bt = 0, Dn = 0, L = 0;
    bool bf16 = false;
    bool vec_ok = false;             // rows of every (Bt, Dn, L) tensor are whole aligned 16-byte vectors
};

struct GatedUpdateLaunch {
    float* state;                    // (Bt, Dn), in/out
    const void* x;
    const void* f;
    const void* i;
    const float* rate;
    void* out;
    int64_t Dn, R;                   // R = Bt * Dn
    bool bf16;
};
// Scratch floats of the forward and the backward, by sizes alone.
int64_t gated_fwd_scratch(int64_t Bt, int64_t Dn, int64_t L);
int64_t gated_bwd_scratch(int64_t Bt, int64_t Dn, int64_t L);
hipError_t launch_gated_fwd(const GatedLaunch& a, hipStream_t stream);
hipError_t launch_gated_bwd(const GatedLaunch& a, hipStream_t stream);
hipError_t launch_gated_update(const GatedUpdateLaunch& a, hipStream_t stream);

// Causal conv1d's gradients (conv1d_bwd.hip).
struct ConvBwdLaunch {
    const void* x;
    const float* w;
    const float* bias;      // nullable
    const void* state_in;   // (Bt, Dn, K-1), nullable
    const void* dout;
    const void* dfinal;     // (Bt, Dn, K-1), nullable
    void* dx;
    float* dw;              // (Dn, K)
    float* db;              // nullable
    void* dstate;           // (Bt, Dn, K-1), nullable
    float* scratch;
    int64_t Dn, L, R;       // R = Bt * Dn
    int K;
    bool silu, bf16;
    bool vec_ok;            // rows of x / dout / dx are whole aligned 16-byte vectors
};
int64_t conv1d_bwd_scratch(int64_t Bt, int64_t Dn, int64_t L, int64_t K);
hipError_t launch_conv1d_bwd(const ConvBwdLaunch& a, hipStream_t stream);

// Beam search (beam.hip).
constexpr int kBeamMost = 64;     // beams, and continuations kept, per request
constexpr int kReorderMost = 64;  // state tensors per launch

struct BeamSelectLaunch {
    const void* logits;           // (Bt, N, V)
    const float* scores;          // (Bt, N)
    const int32_t* finished;      // (Bt, N), nullable
    float* next_scores;           // (Bt, K)
    int32_t* parents;
    int32_t* tokens;
    int32_t* next_finished;       // nullable
    float* scratch;
    int64_t Bt, N, V, K;
    int end;                      // -1: no end token
    bool bf16, vec_ok;            // rows of logits are whole aligned 16-byte vectors
};
struct BeamReorderLaunch {
    void* data;
    int64_t bytes;                // of one beam's state
};
int64_t beam_select_scratch(int64_t Bt, int64_t N, int64_t V, int64_t K);
hipError_t launch_beam_select(const BeamSelectLaunch& a, hipStream_t stream);
hipError_t launch_beam_reorder(const BeamReorderLaunch* states, int count, const int32_t* parents, int64_t Bt, int N,
                               hipStream_t stream);

// RMS norm (rms_norm.hip): rows of W columns.
constexpr int64_t kNormWidest = 16384;

struct NormLaunch {
    const void* x;
    const void* residual;        // nullable
    const float* weight;
    void* out;                   // the type of x; e4m3 with scales
    void* residual_out;          // with residual
    float* rstd;                 // (R), nullable
    float* scales;               // (R, G), nullable
    int64_t R, W;
    float eps;
    int G;                       // 1, or ceil(W / 128)
    bool x_bf16, residual_bf16;
    bool vec_ok;                 // rows of every tensor are whole aligned 16-byte vectors (8-byte ones in e4m3)
};
struct NormBwdLaunch {
    const void* z;
    const float* weight;
    const float* rstd;
    const void* dout;
    const void* dresidual_out;   // nullable
    void* dx;                    // the type of dout
    void* dresidual;             // the type of z, nullable
    float* dweight;              // nullable
    float* scratch;              // with dweight
    int64_t R, W;
    bool x_bf16, z_bf16, vec_ok;
};
int64_t rms_norm_bwd_scratch(int64_t R, int64_t W);
hipError_t launch_rms_norm_fwd(const NormLaunch& a, hipStream_t stream);
hipError_t launch_rms_norm_bwd(const NormBwdLaunch& a, hipStream_t stream);

// Linear attention (linear_attention.hip): rows (Bt, L, heads, dim), states (Bt, H, K, V).
constexpr int kAttnMostDim = 128;

struct AttnLaunch {
    const void* q;               // (Bt, L, Hq, K)
    const void* k;               // (Bt, L, Hk, K)
    const void* v;               // (Bt, L, Hv, V)
    const float* rate;           // (H)
    const float* h0 = nullptr;   // nullable
    const int32_t* lens = nullptr;  // (Bt), nullable
    void* out = nullptr;         // (Bt, L, H, V), nullable
    float* last_state = nullptr; // nullable
    // the backward's
    const void* dout = nullptr;  // (Bt, L, H, V)
    const float* dlast = nullptr;   // nullable
    void* dq = nullptr;
    void* dk = nullptr;
    void* dv = nullptr;
    float* dh0 = nullptr;        // nullable
    float* scratch = nullptr;
    int64_t Bt = 0, L = 0;
    int H = 0, Hq = 0, Hk = 0, Hv = 0, K = 0, V = 0;
    float scale = 1.0f;
    bool bf16 = false;
};
struct AttnUpdateLaunch {
    float* state;                // (Bt, H, K, V), in/out
    const void* q;               // (Bt, Hq, K)
    const void* k;               // (Bt, Hk, K)
    const void* v;               // (Bt, Hv, V)
    const float* rate;
    void* out;                   // (Bt, H, V)
    int64_t Bt;
    int H, Hq, Hk, Hv, K, V;
    float scale;
    bool bf16;
};
int64_t attn_fwd_scratch(int64_t Bt, int64_t L, int H, int K, int V, bool bf16);
int64_t attn_bwd_scratch(int64_t Bt, int64_t L, int H, int Hq, int Hk, int Hv, int K, int V, bool bf16);
hipError_t launch_attn_fwd(const AttnLaunch& a, hipStream_t stream);
hipError_t launch_attn_bwd(const AttnLaunch& a, hipStream_t stream);
hipError_t launch_attn_update(const AttnUpdateLaunch& a, hipStream_t stream);

// Token log probabilities (token_logprobs.hip): rows of V logits.
struct LogprobLaunch {
    const void* logits;          // (R, V)
    const int32_t* tokens;       // (R)
    float* logprobs;             // (R)
    float* entropy;              // (R), nullable
    float* top_logprobs;         // (R, K), nullable
    int32_t* top_tokens;         // (R, K)
    float* saved;                // (R, 3), nullable
    float* scratch;
    int64_t R, V;
    int K;                       // 0: no alternatives
    bool bf16;
};
struct LogprobBwdLaunch {
    const void* logits;
    const int32_t* tokens;
    const float* saved;
    const float* dlogprobs;      // (R)
    const float* dentropy;       // (R), nullable
    void* dlogits;               // (R, V); may be logits
    int64_t R, V;
    bool bf16, vec_ok;
};
int64_t logprob_scratch(int64_t R, int64_t V, int64_t K);
hipError_t launch_logprob_fwd(const LogprobLaunch& a, hipStream_t stream);
hipError_t launch_logprob_bwd(const LogprobBwdLaunch& a, hipStream_t stream);

}  // namespace mss
