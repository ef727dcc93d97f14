// QK norm and rotary positions: how a call is shared out, its launches, and the sums of the weights'
// gradients (the kernel: qk_rope.cuh).
#include "qk_rope.cuh"

namespace slra {
namespace {

// The weights' gradients: the workers' sums joined in a fixed order, 32 columns a cluster.
__global__ void __launch_bounds__(32 * kFinalWarps) qk_rope_final_kernel(const float* part, int workers, int columns,
                                                                         int q_columns, float* dwq, float* dwk, int splits) {
    __shared__ float red[kFinalWarps][32], total[1][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x / splits * 32 + lane;
    float sum[1] = {0.f};
    wait_for_rows();
    if (c < columns)
#pragma unroll 8
        for (int w = warp + blockIdx.x % splits * kFinalWarps; w < workers; w += kFinalWarps * splits)
            sum[0] += part[static_cast<long long>(w) * columns + c];
    red[warp][lane] = sum[0];
    __syncthreads();
    if (warp == 0) {
        sum[0] = 0.f;
        for (int w = 0; w < kFinalWarps; ++w) sum[0] += red[w][lane];
        total[0][lane] = sum[0];
    }
    if (splits > 1) join_cluster<1>(total, sum, splits);
    if (warp != 0 || c >= columns || blockIdx.x % splits != 0) return;
    if (c < q_columns) {
        if (dwq) dwq[c] = sum[0];
    } else if (dwk) {
        dwk[c - q_columns] = sum[0];
    }
}

// Threads of a head, rounded up to what a warp's exchanges sum over.
int even_group(int head_dim) {
    int g = 1;
    while (g * 8 < head_dim) g *= 2;
    return g;
}

// A block takes all heads of a token, a part of q's and of k's (no norm, or one per head), or q's or k's alone
// (they never share a norm), whichever costs the fewest thread-steps by the rule below.  The rule against the
// clock: 12 + 12 heads of 128 forward together 78 us, apart 107, two vectors a thread apart 123; backward apart
// 187, together 197; 32 + 8 heads forward with two vectors of q and one of k 127 us, one of each 199, backward
// 367 and 393 (apart 504).
struct RopePlan {
    RowPlan rows;
    int group, split_sides, part_heads[2];
};

RopePlan plan_of(long long rows, int head_dim, int q_heads, int k_heads, int norm, bool backward) {
    RopePlan best;
    long long least = -1;
    // Threads of a head: as many as it has vectors, so that heads of 80 idle no thread in three, if no norm per head
    // sums over them; else, or where a thread's second vector would not then be at the same place of its head, a
    // power of two.
    for (int G = norm == kQkNormHead ? even_group(head_dim) : head_dim / 8;; G = even_group(head_dim)) {
        // parts of the heads, or sides apart (parts 0); vectors a thread of q and of k, or of the side
        for (int parts = 0; parts <= 16; ++parts) {
            if ((norm == kQkNormToken && parts > 1) || (parts == 0 && !k_heads)) continue;
            const int hq = parts ? (q_heads + parts - 1) / parts : std::max(q_heads, k_heads);
            const int hk = parts ? (k_heads + parts - 1) / parts : 0;
            for (int vq = 1; vq <= 2; ++vq) {
                RopePlan c;
                RowPlan& p = c.rows;
                row_team(std::max((hq * G + vq - 1) / vq, hk * G), 1, &p);
                p.VQ = vq;
                p.V = vq + (hk ? 1 : 0);
                if ((vq > 1 && p.team % G != 0) || p.threads > rope_threads(p.V, backward) || (p.team <= 32 && vq > 1)) continue;
                // Thread-steps of a row: a step costs about as much as two vectors besides its vectors (three with one
                // token a step), and an entry of the table as much as one; times the registers that a thread takes from
                // the SM, between what it needs and its share where the blocks leave some over (the needs alone: 90
                // drawn calls 6% slower, 21,881 x 2 tokens of 23 + 23 heads backward 525 us for 353; the shares alone 1%
                // slower, 32,760 tokens of 12 + 12 heads forward 107 us for 79).  Sides apart cost both blocks the
                // table, and leave threads idle where they are unequal.
                const int needed[2][4] = {{0, 80, 96, 128}, {0, 96, 120, 168}};
                const int blocks = rope_blocks_per_sm(p, backward, norm != kQkNormNone);
                const int registers = needed[backward][p.V] + 65536 / (blocks * p.threads);
                const int steps = backward && p.V > 1 ? 3 : 2;
                const int shares = parts ? parts : 2 * std::min(q_heads, k_heads) < std::max(q_heads, k_heads) ? 3 : 2;
                const long long cost = static_cast<long long>((2 * p.V + steps) * p.team + head_dim) *
                                       registers * shares;
                if (least >= 0 && cost >= least) continue;
                least = cost;
                c.group = G;
                c.split_sides = parts == 0;
                c.part_heads[0] = hq;
                c.part_heads[1] = parts ? hk : hq;
                p.parts = parts ? parts : 2;
                best = c;
            }
        }
        if (G == even_group(head_dim)) break;
    }
    RowPlan& p = best.rows;
    const int parts = p.parts;
    row_workers(rows, std::max(1, kSMs * rope_blocks_per_sm(p, backward, norm != kQkNormNone) / parts), &p);
    p.parts = parts;
    p.blocks *= parts;
    return best;
}

}  // namespace

RowPlan qk_rope_plan(long long rows, int head_dim, int q_heads, int k_heads, int norm, bool backward) {
    return plan_of(rows, head_dim, q_heads, k_heads, norm, backward).rows;
}

cudaError_t launch_qk_rope(const QkRopeArgs& args, bool backward, cudaStream_t st) {
    QkRopeArgs a = args;
    const RopePlan plan = plan_of(a.rows, a.head_dim, a.side[0].heads, a.side[1].heads, a.norm, backward);
    const RowPlan& p = plan.rows;
    a.parts = p.parts;
    a.split_sides = plan.split_sides;
    a.part_heads[0] = plan.part_heads[0];
    a.part_heads[1] = plan.part_heads[1];
    a.group = plan.group;
    a.team = p.team;
    a.workers = p.workers;
    a.share = p.share;
    const bool all = a.rotated == kRopeAll;
    const auto launch = !backward               ? (all ? launch_qk_rope_fwd : launch_qk_rope_fwd_some)
                        : a.norm == kQkNormNone ? (all ? launch_qk_rope_bwd_none : launch_qk_rope_bwd_none_some)
                        : a.norm == kQkNormHead ? (all ? launch_qk_rope_bwd_head : launch_qk_rope_bwd_head_some)
                                                : (all ? launch_qk_rope_bwd_token : launch_qk_rope_bwd_token_some);
    const cudaError_t e = launch(a, p, st);
    if (e != cudaSuccess || !backward || !a.part) return e;
    const bool each = a.norm == kQkNormToken;  // a weight of its own for each head
    const int q_columns = a.head_dim * (each ? a.side[0].heads : 1);
    const int k_columns = a.head_dim * (each ? a.side[1].heads : a.side[1].heads > 0);
    const int columns = q_columns + k_columns;
    const int workers = each ? p.workers : p.workers * p.parts;
    const int splits = join_splits(workers, (columns + 31) / 32);
    return launch_join(qk_rope_final_kernel, (columns + 31ll) / 32 * splits, splits, st, a.part, workers, columns, q_columns,
                       a.side[0].dweight, a.side[1].dweight, splits);
}

}  // namespace slra
