// Gradients of the norm after a block (ssd_block_norm_kernel's formula) and of the gate and grouped norm after the scan:
//   ssd_block_norm_bwd_kernel   p2 = next_weight dout, hh = h rstd2:  dh = dres + rstd2 (p2 - hh mean(p2 hh))
//   (_loose: odd alignments)    p1 = scale dh weight,  uh = u rstd1:  du = rstd1 (p1 - uh mean(p1 uh))
//                               dx = du silu(gate),  dgate = du x s (1 + gate (1 - s)),  s = 1 / (1 + e^-gate)
//                               and each row slot's shares of  dweight = sum scale dh uh,  dnext_weight = sum dout hh
//   (without a residual: scale dh is dout itself)
//
// u and both rstd are recomputed from x, gate and h, which may be 8-bit rows.  A grid as large as the GPU holds at
// once walks the rows, so that the shares stay few; ssd_share_sum adds them in a fixed order.
//
// Up to five operands a row are too many to keep the next row's in registers, and HBM wants some 50 KB in flight per
// SM.  So each thread copies its own vectors of the rows to come into its warp's records in shared memory (cp.async), up to
// three rows ahead, or with a residual as soon as a row's operands are read for the last time: no barrier and no register holds
// them, and each pass over the row reads them there.  The weights lie there too.  What the kernel runs out of first is issue
// slots: arithmetic is on pairs of numbers, and a record's pieces lie at constant offsets.
//
// Times with the shares' sum (7 us of them), and parts of the copy's rate: gate and norm 16384 x 5120 bf16 140 us, 89 %; from 8 bits
// 12289 x 5120, with the result computed again, 123 us, 76 % (issue slots 57 % busy, shared memory's and the stores' wavefronts 62 %:
// codes are decoded and the weights read in both passes); with a residual in fp32 16384 x 2560 155 us, 88 % (163 us while x was asked
// for after the last pass); all operands in 8 bits 9001 x 1533 69 us, 39 % (1536 columns 52 us).  There neither HBM nor the issue slots
// (54 %) are full: h is decoded in passes one and two, x in two and three, the gate once, and a CTA's next row, 10.7 KB, is
// asked for after the second pass only; at 1533 columns 97 of 128 threads have any, and first and last
// vectors go by elements.
#include "ssd_block_norm_bwd.cuh"

namespace ssd {

// Enough for every shape: which one a call takes depends on its addresses and types too.
int64_t block_norm_bwd_lines(int64_t rows, int size, int groups) {
    const RowPlan loose = loose_plan(rows, size, groups);
    int most = loose.slots + loose.late_slots;
    for (int narrow : {kNarrowSpan, kNarrowSpanLong})
        for (int span : {size, vector_span(size)}) {
            RowPlan p = vector_plan(span, narrow);
            for (int per_sm = ctas_sm(p.threads, threads_sm(p.elems, false)); per_sm > 0; --per_sm) {
                spread(p, rows, groups, per_sm, true);
                if (p.slots + p.late_slots > most) most = p.slots + p.late_slots;
            }
        }
    return most / groups;
}

cudaError_t launch_gate_norm_bwd_typed(BlockNormBwdArgs& a, int* lines, cudaStream_t st) {
    return a.dtype == SSD_BF16 ? launch_block_norm_bwd_typed<bf16_t, bf16_t, true, false>(a, lines, st)
                               : launch_block_norm_bwd_typed<float, float, true, false>(a, lines, st);
}

cudaError_t launch_block_norm_bwd(const BlockNormBwdArgs& args, cudaStream_t st) {
    BlockNormBwdArgs a = args;
    a.inv_size = 1.f / (float)a.size;
    int lines = 0;
    const cudaError_t e = !a.dres                          ? launch_gate_norm_bwd_typed(a, &lines, st)
                          : a.dtype == SSD_F32             ? launch_block_norm_bwd_f32(a, &lines, st)
                          : a.residual_dtype == SSD_F32    ? launch_block_norm_bwd_bf16_f32(a, &lines, st)
                                                           : launch_block_norm_bwd_bf16(a, &lines, st);
    if (e != cudaSuccess) return e;
    const int width = a.size * a.groups;
    return launch_share_sum(a.shares, lines, width, a.next_weight ? 2 * width : width, a.dweight, a.dnext_weight, false, st);
}

}  // namespace ssd
