// ssm.h -- launch parameters and launchers of the state space layer's kernels (host side):
// short causal convolution, selective scan, gated row norm, each as declared in
// include/ramnet.h.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace ramnet {

struct ConvParams {
    const void* x;  // element (b, t, c) at b*sb + t*st + c
    int64_t sb, st;
    int in_bf16;
    const float* w;         // [C,W]
    const float* bias;      // [C] or null
    int silu;
    const int32_t* lengths;  // [B] or null (all T)
    const void* state_in;    // [B,W-1,C] or null (zeros)
    void* y;                 // [B,T,C]
    int out_bf16;
    void* state_out;  // [B,W-1,C] or null; may alias state_in
    int B, T, C, W;
    uint32_t* status;
};

struct ConvStepParams {
    const void* x;  // element (b, c) at b*sb + c
    int64_t sb;
    int in_bf16;
    const float* w;
    const float* bias;
    int silu;
    void* state;  // [B,W-1,C], shifted in place
    void* y;      // [B,C]
    int out_bf16;
    int B, C, W;
    uint32_t* status;
};

// Element strides of one [B,T,H,.] operand (last dimension contiguous).
struct Str3 {
    int64_t b, t, h;
};

// How the prompt form cuts each sequence: `nseg` segments of `seg_len` tokens run side by side.  A
// first launch finds what each piece of the sequence before the last segment adds to a zero state
// (`sub` pieces per segment), a second chains these into the states the segments start from, and
// the third computes the outputs.  With one segment only the third launch runs.
struct SsmSplit {
    int nseg, seg_len, sub;
    __host__ __device__ int pieces() const { return (nseg - 1) * sub; }
    __host__ __device__ int piece_len() const { return seg_len / sub; }
    __host__ __device__ int slots() const { return pieces() + 1; }  // states per (sequence, head) in the workspace
};

// Step sizes and decays of 64 tokens of one head, for the tensor-core form.  With a_i the sum of d A over the
// chunk's tokens up to i, in powers of two (times log2 e); blocks are 16 tokens.
struct ChunkTok {
    float hi[64], lo[64];  // a_i as the sum of two floats
    float d[64];           // step sizes
    float ein[64];         // 2^a_i
    float w[64];           // 2^(a_63 - a_j) d_j
    float u[64];           // 2^(a_i - sum before i's block)
    float v[64];           // 2^(sum up to the end of j's block - a_j) d_j
    float dec;             // 2^a_63
    float blk[3];          // 2^ the sums of blocks 1 and 2, and of both
    double total, pad;     // a_63
};
constexpr int kChunk = 64;
constexpr int kWaitNs = 2000000000;  // default limit of a wait
constexpr int kPollNs = 4000;        // a poll of a barrier that is not there yet, suspended by the hardware (measured)

struct SsmParams {
    const void* x;  // [B,T,H,P]
    Str3 xs;
    const void* dt;  // [B,T,H]
    Str3 dts;
    const float* A;  // [H]
    const void* Bm;  // [B,T,G,N]
    Str3 bs;
    const void* Cm;  // [B,T,G,N]
    Str3 cs;
    int in_bf16;
    const float* D;          // [H] or null
    const float* dt_bias;    // [H] or null
    const int32_t* lengths;  // [B] or null
    const float* S_in;       // [B,H,N,P] or null
    void* y;                 // [B,T,H,P]
    int out_bf16;
    float* S_out;  // [B,H,N,P]
    int B, T, H, G, N, P;
    int softplus;
    float dt_min, dt_max;
    SsmSplit split;
    float* seg_state;  // [B,H,slots,N,P]: what piece i adds; then, in slot k*sub, the state segment k starts from
    float* seg_decay;  // [B,H,pieces]
    ChunkTok* toks;    // [B,H,ceil(T/64)], the tensor-core form only
    uint32_t* status;
    int poll_cost;  // of a wait of the tensor-core form: what one poll takes of the kWaitNs that it may last
};

struct SsmStepParams {
    const void* x;  // [B,H,P]
    Str3 xs;
    const void* dt;  // [B,H]
    Str3 dts;
    const float* A;
    const void* Bm;  // [B,G,N]
    Str3 bs;
    const void* Cm;
    Str3 cs;
    int in_bf16;
    const float* D;
    const float* dt_bias;
    float* S;  // [B,H,N,P], updated in place
    void* y;   // [B,H,P]
    int out_bf16;
    int B, H, G, N, P;
    int softplus;
    float dt_min, dt_max;
    uint32_t* status;
};

struct NormParams {
    const void* x;  // element (r, d) at r*sx + d
    int64_t sx;
    const void* z;  // or null
    int64_t sz;
    int in_bf16;
    const float* w;  // [D] or null (ones)
    void* y;         // [R,D]
    int out_bf16;
    int64_t R;
    int D, groups;
    float eps;
    int gate_first;
    uint32_t* status;
};

// Device address of the library's status word on the current device (null on a CUDA error).
uint32_t* library_status_word();
// Limit of each wait of a prompt's kernels (ramnet_set_scan_wait_limit), at most kWaitNs.
int scan_wait_ns();

cudaError_t launch_conv(const ConvParams& p, cudaStream_t stream);
cudaError_t launch_conv_step(const ConvStepParams& p, cudaStream_t stream);
cudaError_t launch_ssm_step(const SsmStepParams& p, cudaStream_t stream);
cudaError_t launch_norm_gate(const NormParams& p, cudaStream_t stream);

// How sequences are cut by the tensor-core form and by the token-by-token form (launch_ssm_scan sets p.split).
SsmSplit ssm_split(int B, int T, int H, int G, int P);
SsmSplit ssm_split_plain(int B, int T, int H, int N, int P);
cudaError_t launch_ssm_scan(const SsmParams& p, cudaStream_t stream);
cudaError_t launch_ssm_chain(const SsmParams& p, cudaStream_t stream);
// The tensor-core form, for the types, sizes and layouts it takes.
bool ssm_mma_takes(const SsmParams& p);
cudaError_t launch_ssm_mma(const SsmParams& p, cudaStream_t stream);

}  // namespace ramnet
