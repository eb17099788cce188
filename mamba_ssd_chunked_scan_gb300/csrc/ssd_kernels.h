// Host-side declarations shared by the libssd CUDA sources.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssd {

struct WsHeader;

enum { kModeFull = 0, kModeAggregate = 1 };

// Polls a device-side wait of the tensor-core kernels makes before it gives up
// (each poll is an mbarrier try_wait, which may suspend the thread for a while;
// every wait also gives up after 2 s).
constexpr uint32_t kDefaultWaitIters = 1u << 26;
// Smallest wait cap the fault-injection entry points accept: the drain waits
// share the cap and must outlast the MMAs and copies still in flight.
constexpr uint32_t kMinInjectWaitRounds = 4096;

// Everything one launch of a chunk kernel needs (passed by value).
struct FwdArgs {
    int64_t batch, L;
    int H, P, N, G;
    int Q;                 // chunk the kernel uses
    int64_t split_len;     // tokens per split (== L rounded up when one split)
    int nsplit;
    int dtype;             // ssd_dtype_t
    int mode;              // kModeFull or kModeAggregate
    const void* x;
    const float* dt;
    const float* A;
    const void* B;
    const void* C;
    const float* D;
    const float* init;
    const int32_t* cu;
    int ndocs;
    void* y;
    float* fin;
    float* ws_tau;         // [batch * H * nsplit] natural-log split decays
    float* ws_state;       // [batch * H * nsplit * P * N] split aggregates (slot s); after the
                           // scan, slot s - 1 holds the state entering split s
    WsHeader* ws;
    // n / H, n / nsplit and n / (H / G) for 0 <= n < 2^31 as (mulhi(m, n) + n) >> l
    uint32_t divH_m, divH_l, divS_m, divS_l, divHG_m, divHG_l;
    // leftover-unit plan (tail_units > 0, one split otherwise): the (row, head) units
    // [0, tail_first) run whole, the last tail_units are cut into nsplit pieces of
    // split_len tokens; grid_units = CTAs of this launch (0: batch * H * nsplit)
    int tail_units;
    int64_t tail_first;
    int64_t grid_units;
    // bounded waits give up after this many polls (kDefaultWaitIters) or 2 s
    uint32_t wait_iters;
    // fault injection (test aid, 0 otherwise): the TMA producer issues no loads,
    // so every wait that depends on them runs out
    int stall_loads;
    // launched as a programmatic dependent of the call's previous launch (tensor-core
    // full pass, split scan, document-start aggregates)
    int pdl;
};

// One decode step (ssd_step): everything the launch needs.
struct StepArgs {
    int64_t batch;
    int H, P, N, G;
    int dtype;             // ssd_dtype_t of x, B, C and y
    const float* state_in;
    float* state_out;      // == state_in for an in-place step
    const void* x;
    const float* dt;
    const float* A;
    const void* B;
    const void* C;
    const float* D;
    void* y;
};

// Backward pass (ssd_bwd): everything its two launches need.
struct BwdArgs {
    int64_t batch, L;
    int H, P, N, G;
    int Qb;                // backward chunk (tokens)
    int dtype;             // ssd_dtype_t of x, B, C, dy, dx, dB, dC
    const void* x;
    const float* dt;
    const float* A;
    const void* B;
    const void* C;
    const float* D;
    const float* init;
    const void* dy;
    const float* dfin;
    const int32_t* cu;     // packed documents (batch 1), or NULL
    int ndocs;
    void* dx;
    float* ddt;
    float* dA;
    void* dB;
    void* dC;
    float* dD;
    float* dinit;
    float* ws_ckpt;        // [batch * H * nchunks * P * N] state entering each chunk
    float* ws_dB;          // [batch * L * H * N] per-head shares of dB (fp32, or bf16: shares_bf16)
    float* ws_dC;          // [batch * L * H * N] per-head shares of dC
    int shares_bf16;       // the shares are bf16 (the tensor-core backward)
    float* ws_dA;          // [batch * H]
    float* ws_dD;          // [batch * H]
    WsHeader* ws;          // status word (the tensor-core kernel's bounded waits)
    // sequence splits of the tensor-core backward (nsplit 1: whole rows); units are
    // (b * H + h) * nsplit + s, and ws_dA / ws_dD hold one share per unit (the
    // CUDA-core kernel with packed documents: nsplit = ndocs, units h * ndocs + d)
    int nsplit;
    int64_t split_len;     // tokens per split, a multiple of 128
    const float* ws_sin;   // [batch * H * nsplit * P * N] slot s - 1: the state entering split s
    const float* ws_lam;   // [batch * H * nsplit * P * N] slot s + 1: the adjoint of the state leaving split s
    uint32_t wait_iters;   // poll cap of each bounded wait (0: the default)
    // packed documents with their own states on the tensor cores: units h * ndocs + d
    // (nsplit = ndocs), each document in chunks from its first token; ws_ckpt holds
    // L / 128 + ndocs chunks per head
    int doc_units;
};

// Gated RMS normalisation (ssd_gate_norm): everything its launch needs.
struct GateNormArgs {
    int64_t rows;
    int width, group_size;
    int dtype;             // ssd_dtype_t of y, z and out
    float eps;
    const void* y;
    const void* z;
    const float* weight;
    void* out;
};

// Residual RMS norm (ssd_add_norm) and its gradient (ssd_add_norm_bwd).
constexpr int kAddNormMaxWidth = 16384;   // 1024 threads x 16 elements
constexpr int kAddNormSMs = 152;          // SMs the backward's row slots (and its workspace) are sized for
struct AddNormArgs {
    int64_t rows;
    int width;
    int dtype, residual_dtype, out_dtype;
    float eps;
    const void* x;
    const void* residual;  // or NULL
    const float* weight;
    void* out;
    float* scales;         // e4m3 out: [rows]
    void* residual_out;    // or NULL
    float* rstd;           // [rows], or NULL
    int rows_per_cta;
};
struct AddNormBwdArgs {
    int64_t rows;
    int width;
    int dtype, residual_dtype;
    const void* dout;
    const void* h;
    const float* weight;
    const float* rstd;
    const void* dres;      // or NULL
    void* dx;              // dtype, or NULL
    void* dres_out;        // residual_dtype, or NULL
    float* dweight;
    float* shares;         // [row slots * width]
    int rows_per_cta;
    float inv_width;
};

// 8-bit rows (ssd_pack_rows, ssd_unpack_rows): units are rows' groups of columns.
constexpr int kPackMaxSize = 16384;   // 1024 threads x 16 elements
struct PackArgs {
    int64_t units;         // rows * groups
    int size;              // columns of a unit
    int groups;
    int dtype;             // of x or out
    int64_t stride;        // elements between rows of x (packing) or of the codes (unpacking)
    const void* x;
    void* codes;
    float* scales;         // [units]
    void* out;
    bool power_only;       // unpacking: by the scales' powers of two alone (their factors are elsewhere)
    int units_per_cta;
};

// The norm after a block (ssd_block_norm) and the gate and norm after the scan with its checkpoint (ssd_gate_norm_pack), and their
// gradients.  Units are rows, or rows' groups of columns (gate and norm; no residual then).
constexpr int kBlockNormMaxSize = 8192;   // 512 threads x 16 elements
struct BlockNormArgs {
    int64_t units;         // rows * groups
    int size;              // columns of a unit
    int groups;
    int dtype, residual_dtype, out_dtype;
    int64_t gate_stride;   // elements between rows of gate
    float scale, eps;
    const void* x;
    const void* gate;      // or NULL
    const void* residual;  // or NULL: out is the first norm's result
    const float* weight;
    const float* next_weight;   // or NULL: no second norm
    void* residual_out;
    void* out;
    float* out_scales;     // e4m3 out: [units]
    void* x_codes;         // or NULL: nothing is kept
    float* x_scales;
    void* gate_codes;
    float* gate_scales;
    // set at the launch: slots (a number of rows at a time, each of its groups), those of a CTA, rows on their way in shared memory
    uint32_t slots;
    int units_per_cta, stages;
    float inv_size;
};
struct BlockNormBwdArgs {
    int64_t rows;
    int size, groups;
    int dtype, residual_dtype;
    int64_t gate_stride, dgate_stride;
    float scale, eps;
    const void* dout;      // NULL: no second norm
    const void* dres;      // NULL: no residual
    const void* x;         // of dtype, or codes where it has scales; gate and h so too
    const float* x_scales;
    const void* gate;      // or NULL
    const float* gate_scales;
    const void* h;
    const float* h_scales;
    const float* weight;
    const float* next_weight;
    void* dx;
    void* dgate;
    void* dres_out;
    void* out;             // the forward's, or NULL (gate and norm)
    float* dweight;
    float* dnext_weight;
    float* shares;         // [share_lines * width * weights]
    int64_t share_lines;   // a launch that would leave more is refused
    // set at the launch: the rows' slots, and their shared memory (weights, then stages of operands and scales)
    int slots, late_slots, early_rows, slots_per_cta;
    int stages;
    float inv_size;
};

// Gated linear recurrence (ssd_gate_scan, ssd_gate_scan_bwd): tiles of kScanSegs segments x kScanCh
// channels.  A segment holds as many tokens as let two tiles' values stay in a thread's registers (one exp(-g)
// per element forwards, two values backwards) and three or four tiles' operands in shared memory; fewer where
// rows are off 16-byte alignment (two values forwards too).
// A state is handed over once per kScanBlock tiles of a sequence.
constexpr int kScanSegs = 16, kScanCh = 64, kScanBlock = 16, kScanMinTok = 64;
constexpr int scan_seg(bool bwd, int dtype, bool rows) {
    return dtype == 1 /* SSD_BF16 */ ? (bwd || rows ? 8 : 16) : (bwd || rows ? 4 : 8);
}
struct GateScanArgs {
    int64_t batch, seqlen;
    int width;
    int dtype;
    int64_t g_stride, x_stride;   // elements between tokens of g, dg and of x, dx
    int ndocs;
    const void* g;
    const void* x;
    const float* init;
    const int32_t* cu;
    void* y;               // forward: written; backward: the forward's output
    const void* dy;
    void* dg;
    void* dx;
    // per row or document, what enters the walk and what leaves it: initial and final states forwards,
    // the final states' and the initial states' gradients backwards
    const float* enter;
    float* leave;
    // fault injection: bounded waits give up after so many polls (0: an ordinary call); tiles that a CTA loads before it stalls
    // (negative: all), or no tile publishes its map
    uint32_t wait_iters;
    int loads, mute;
    // set at the launch
    WsHeader* ws;
    uint32_t* ticket;
    uint64_t* maps;        // per tile and channel
    uint64_t* carry;       // per block and channel
    int64_t nchunks;       // tiles along a sequence
    int64_t nblocks;       // blocks of tiles along a sequence
    int ngroups;           // channel groups
    uint32_t ntiles;
};
struct GateScanLayout {    // workspace, in bytes
    int64_t nchunks, nblocks;
    int ngroups;
    size_t ticket_off, maps_off, carry_off, total;
};
struct GateStepArgs {
    int64_t batch;
    int width;
    int dtype;
    int64_t g_stride, x_stride;
    const void* g;
    const void* x;
    const float* state_in;
    float* state_out;
    void* y;
};

// Matrix product with its epilogue (ssd_linear, ssd_linear_bwd): D = X W^T.
constexpr int kLinearSwap = 64;       // up to this many rows of x the product is computed transposed
constexpr int kLinearTileRows = 128;  // of a CTA's tile; a pair's has twice as many
constexpr int kLinearSMs = 152;       // SMs the plan (and so the workspace) is made for
constexpr int kLinearMaxSplits = 16;
struct LinearOperand {
    const void* p;
    int64_t ld;            // elements between its rows in memory
    bool along_rows;       // the contraction runs along its rows (the operand is stored transposed; bf16)
};
struct LinearArgs {
    int64_t m;             // rows of D
    int n;                 // columns of D
    int64_t k;             // contraction
    int dtype;             // of the operands: SSD_BF16 or SSD_E4M3
    int act;               // ssd_act_t
    LinearOperand x, w;
    const float* x_scales; // [m], or NULL
    const float* w_scales; // [n], or NULL
    const float* bias;     // [n], or NULL
    const void* residual;  // (m, n) bf16, or NULL
    void* y;               // (m, n) bf16
    void* pre;             // (m, n) bf16, or NULL
    float* parts;          // per part, a tile of fp32 sums
    WsHeader* ws;
    int keep_status;       // the status word was cleared by the call already
    // fault injection: bounded waits give up after so many polls (0: an ordinary call); blocks of the contraction that a CTA
    // loads before it stalls
    uint32_t wait_iters, loads;
    int swap, vec;         // set at the launch
};
struct LinearPlan {
    int tile_n;
    int64_t whole;         // tiles computed whole; the others in `splits` parts
    int splits;
    bool swap, pair;
    size_t parts_bytes;
};
struct LinearDpreArgs {
    int64_t m;
    int n;
    int act;
    int64_t ldp;
    const void* dy;
    const void* pre;       // or NULL (no activation)
    const float* pre_scales;   // [m]: pre is e4m3 codes; or NULL
    void* dpre;            // (m, ldp) bf16, or NULL
    float* shares;         // [slabs * n], or NULL
    float* dbias;          // [n], or NULL
    int slab_rows;
};
// What comes with x in 8-bit rows.
struct LinearDpreRows {
    const float* x_scales;     // [m], or NULL: dpre is to be multiplied by the factors of these scales (see scale_factor)
    float* inv_factors;        // [m]: their reciprocals, written; or NULL
    float* ones;               // [k]: written; or NULL
    int k;
    PackArgs expand;       // out not NULL: x to be unpacked to bf16 in the same launch, by CTAs from number ctas on
    unsigned ctas;
};

// Constants of division by an invariant divisor d >= 1 through one high
// multiply and a shift (Granlund and Montgomery, "Division by Invariant
// Integers using Multiplication", 1994): l = ceil(log2 d),
// m = floor(2^32 (2^l - d) / d) + 1; then n / d = (mulhi(m, n) + n) >> l,
// exact for 0 <= n < 2^31 (the sum cannot wrap).
inline void fastdiv_consts(uint32_t d, uint32_t* m, uint32_t* l) {
    uint32_t k = 0;
    while ((1ull << k) < d) ++k;
    *l = k;
    *m = (uint32_t)((((1ull << k) - d) << 32) / d + 1);
}

constexpr int kMaxDevices = 256;   // device ordinals the per-device caches cover

// SM count of the current device (cached per device); 0 when no device is visible.
int device_sms();

size_t simt_smem_bytes(int Q, int P, int N);
cudaError_t launch_simt(const FwdArgs& a, cudaStream_t st);
cudaError_t launch_split_scan(const FwdArgs& a, cudaStream_t st);
// 4-D TMA map over a (batch, L, heads_or_groups, inner) bf16 tensor; box = one
// 64-element x 128-row tile of one head (group), 128-byte swizzle.
bool encode_4d(CUtensorMap* tm, const void* base, int64_t inner, int64_t mid, int64_t L, int64_t batch);
size_t tc_smem_bytes();
bool tc_supported(int P, int N, int Q, int dtype);
cudaError_t launch_tc(const FwdArgs& a, cudaStream_t st);
// adds the initial states of packed documents that start inside a split to the
// split aggregates (after the aggregate pass, before their composition)
cudaError_t launch_doc_init_agg(const FwdArgs& a, cudaStream_t st);
int agg_heads_per_cta(int H, int G);
cudaError_t launch_agg_tc(const FwdArgs& a, cudaStream_t st);
cudaError_t launch_agg_rev_tc(const FwdArgs& a, cudaStream_t st);
cudaError_t launch_split_rscan(const FwdArgs& a, const float* dfin, cudaStream_t st);
cudaError_t launch_gate_norm(const GateNormArgs& a, cudaStream_t st);
cudaError_t launch_add_norm(const AddNormArgs& a, cudaStream_t st);
int64_t add_norm_bwd_shares(int64_t rows, int width);   // row slots of the backward
cudaError_t launch_add_norm_bwd(const AddNormBwdArgs& a, cudaStream_t st);
// dw (and next, from column `width` on) = sums over nshares rows of `columns` shares, in a fixed order
cudaError_t launch_share_sum(const float* shares, int nshares, int width, int columns, float* dw, float* next, bool early, cudaStream_t st);
cudaError_t launch_pack(const PackArgs& a, cudaStream_t st);
cudaError_t launch_unpack(const PackArgs& a, cudaStream_t st);
unsigned unpack_flat_ctas(const PackArgs& a);   // CTAs of 256 threads that unpack_flat takes for it; 0: not to be had so
cudaError_t launch_block_norm(const BlockNormArgs& a, cudaStream_t st);
int64_t block_norm_bwd_lines(int64_t rows, int size, int groups);   // rows that the backward's grid walks at once
cudaError_t launch_block_norm_bwd(const BlockNormBwdArgs& a, cudaStream_t st);
size_t gate_scan_workspace(int64_t batch, int64_t seqlen, int width, int dtype);
cudaError_t launch_gate_scan(const GateScanArgs& a, void* workspace, bool bwd, cudaStream_t st);
cudaError_t launch_gate_scan_step(const GateStepArgs& a, cudaStream_t st);
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();   // NULL when the driver has none
LinearPlan linear_plan(int64_t rows, int64_t cols, int64_t kbytes, bool may_swap);
cudaError_t launch_linear(const LinearArgs& a, const LinearPlan& plan, cudaStream_t st);
int64_t linear_dpre_slabs(int64_t m, int n);
cudaError_t launch_linear_dpre(const LinearDpreArgs& a, const LinearDpreRows& x, cudaStream_t st);
size_t bwd_smem_bytes(int Qb, int P, int N);
int bwd_chunk(int P, int N, size_t smem_limit);
cudaError_t launch_bwd(const BwdArgs& a, cudaStream_t st);
// sums the per-head dB, dC shares over each group and the per-row dA, dD shares
cudaError_t launch_bwd_reduce(const BwdArgs& a, cudaStream_t st);
// the backward on the tensor cores: bf16, P = 64, N = 128, chunks of 128 tokens
bool bwd_tc_supported(int P, int N, int dtype);
constexpr int kBwdTcChunk = 128;
cudaError_t launch_bwd_tc(const BwdArgs& a, cudaStream_t st);
size_t step_smem_bytes(int P, int N);
cudaError_t launch_step(const StepArgs& a, cudaStream_t st);
cudaError_t launch_segsum_dump(const float* l2, int64_t nrows, int chunk, float* seg, float* L, float* pexp,
                               float* sfx, cudaStream_t st);

}  // namespace ssd
