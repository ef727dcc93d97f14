// Gated residual and modulated norm: how a call is shared out, its launches, and the sums that several workers
// took part in (the kernels: residual_norm.cuh).
#include "residual_norm.cuh"

namespace slra {
namespace {

// The sums over tokens that more than one worker took part in, joined in a fixed order, 32 channels a warp.
// First the weights' sums, then the modulation rows' (job y counts modulation rows, or the workers' boundaries
// where those are fewer).  A job's partial sums are split over `warps` of a block's, and over the blocks of a
// cluster too where they are many (*_splits: that number of blocks, or 1).
struct Joins {
    int columns, jobs, by_boundary;
    int warps;                    // of a block for a modulation row
    int weight_splits, mod_splits;
    unsigned weight_blocks;       // the first of the modulation rows' blocks
};

__global__ void __launch_bounds__(32 * kFinalWarps)
residual_norm_final_kernel(const __grid_constant__ ResidualNormArgs a, const Joins n) {
    __shared__ float red[3][kFinalWarps][32], total[3][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool weights = blockIdx.x < n.weight_blocks;
    const int splits = weights ? n.weight_splits : n.mod_splits, warps = weights ? kFinalWarps : n.warps;
    const unsigned unit = (weights ? blockIdx.x : blockIdx.x - n.weight_blocks) / splits;
    const int slice = blockIdx.x % splits, c = static_cast<int>(unit % n.columns) * 32 + lane;
    const int job = weights ? 0 : static_cast<int>(unit / n.columns) * (kFinalWarps / warps) + warp / warps;
    bool in = c < a.channels && (weights ? unit < n.columns : job < n.jobs);
    const int rows = static_cast<int>(a.rows);
    // the weights' slots: one a block of the row kernel, its first worker's
    int w0 = 0, w1 = a.blocks - 1, second = -1, g = 0;
    if (!weights && in) {
        g = job;
        if (n.by_boundary) {  // the modulation row that the next worker's first row continues
            const long long r = (job + 1ll) * a.share;
            g = static_cast<int>(r / a.per);
            in = r < rows && r != static_cast<long long>(g) * a.per;
        }
        const int first = g * a.per;
        w0 = first / a.share;
        w1 = (first + a.per - 1) / a.share;
        in = in && w0 != w1;  // else one worker had it all
        // its sums are in the workers' first slots, but in the second one of a worker that came to it from
        // another row
        if (w0 * a.share < first) second = w0;
    }
    float sum[3] = {0.f, 0.f, 0.f};
    wait_for_rows();
    if (in) {
        const long long row = 3ll * a.channels;
#pragma unroll 8
        for (int w = w0 + warp % warps + slice * warps; w <= w1; w += warps * splits) {
            const float* p = weights ? a.wpart + static_cast<long long>(w) * a.teams * row + c
                                     : a.part + (2ll * w + (w == second ? 1 : 0)) * row + c;
#pragma unroll
            for (int k = 0; k < 3; ++k) sum[k] += p[static_cast<long long>(k) * a.channels];
        }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) red[k][warp][lane] = sum[k];
    __syncthreads();
    if (warp % warps == 0) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            sum[k] = 0.f;
            for (int w = 0; w < warps; ++w) sum[k] += red[k][warp + w][lane];
            if (warp == 0) total[k][lane] = sum[k];
        }
    }
    if (splits > 1) join_cluster<3>(total, sum, splits);
    if (warp % warps != 0 || !in || slice != 0) return;
    auto value = [&](const void* p, float fill) {
        if (!p) return fill;
        if (a.w_dtype == kF32) return static_cast<const float*>(p)[c];
        if (a.w_dtype == kBf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[c]);
        return __half2float(static_cast<const __half*>(p)[c]);
    };
    if (weights) {
        if (a.dweight) a.dweight[c] = sum[0];
        if (a.dbias) a.dbias[c] = sum[1];
        if (a.dpost) a.dpost[c] = sum[2];
    } else {
        const long long at = static_cast<long long>(g) * a.channels + c;
        if (a.dshift) a.dshift[at] = sum[0];
        if (a.dscale) a.dscale[at] = value(a.weight, 1.f) * sum[1] + value(a.bias, 0.f) * sum[0];
        if (a.dgate) a.dgate[at] = value(a.post_weight, 1.f) * sum[2];
    }
}

}  // namespace

RowPlan residual_norm_plan(long long rows, int channels, bool backward, bool post, bool token, bool half) {
    RowPlan p;
    p.sums = post && !token;
    const int slots = channels / 8;
    // Two vectors a thread above 5120 channels.  In the backward also where two blocks an SM then hold the rows that
    // only one would else, with 16-bit rows and enough of them (all us, one vector and two): 11,575 x 5 x 3344 with
    // the norm behind the block 756 and 569, 12,665 x 5 x 3056 without 484 and 413, 25,043 x 2 x 3864 with vectors for
    // each token 2220 and 1664.  Not so few rows (1010 x 5 x 2712: 67 and 79), vectors for each token without the norm
    // behind the block (21,853 x 3 x 2952: 1443 and 1719), or an fp32 stream (2900 x 3640: 80 and 90).
    const bool pairs = backward && half && (post || !token) && rows >= 40 * kSMs && slots <= 512 &&
                       slots > bwd_threads(1, p.sums) / 2;
    row_team(slots, slots > 640 || pairs ? 2 : 1, &p);
    row_workers(rows, kSMs * blocks_per_sm(p, backward), &p);
    return p;
}

cudaError_t launch_residual_norm(const ResidualNormArgs& args, bool backward, cudaStream_t st) {
    ResidualNormArgs a = args;
    const RowPlan p = residual_norm_plan(a.rows, a.channels, backward, a.post != kNormNone, a.per == 1, a.stream_dtype != kF32);
    a.team = p.team;
    a.workers = p.workers;
    a.share = p.share;
    a.blocks = p.blocks;
    a.teams = p.threads / p.team;
    const bool token = a.per == 1;  // a modulation row for each row
    const cudaError_t e = backward ? (token ? launch_residual_norm_bwd_token(a, p, st) : launch_residual_norm_bwd(a, p, st))
                                   : (token ? launch_residual_norm_fwd_token(a, p, st) : launch_residual_norm_fwd(a, p, st));
    if (e != cudaSuccess || !backward) return e;
    const long long mods = a.rows / a.per;
    Joins n{};
    n.by_boundary = mods > p.workers ? 1 : 0;
    const bool whole = a.share % a.per == 0 || a.share >= a.rows;  // no modulation row has more than one worker
    n.jobs = a.part && !whole ? static_cast<int>(n.by_boundary ? p.workers - 1 : mods) : 0;
    if (n.jobs == 0 && !a.wpart) return cudaSuccess;
    n.columns = (a.channels + 31) / 32;
    const long long most = n.jobs ? std::min<long long>(a.per / a.share + 2, a.workers) : 0;
    n.weight_splits = a.wpart ? join_splits(a.blocks, n.columns) : 1;
    n.mod_splits = join_splits(most, 1ll * n.columns * n.jobs);
    const int splits = std::max(n.weight_splits, n.mod_splits);
    if (n.weight_splits > 1) n.weight_splits = splits;
    if (n.mod_splits > 1) n.mod_splits = splits;
    n.warps = n.mod_splits > 1 ? kFinalWarps : 1;  // a few partial sums for each
    while (n.warps < kFinalWarps && 6 * n.warps < most) n.warps *= 2;
    const auto clusters = [&](long long blocks) { return (blocks + splits - 1) / splits * splits; };
    n.weight_blocks = a.wpart ? static_cast<unsigned>(clusters(1ll * n.columns * n.weight_splits)) : 0;
    const long long groups = (n.jobs * static_cast<long long>(n.warps) + kFinalWarps - 1) / kFinalWarps;
    return launch_join(residual_norm_final_kernel, n.weight_blocks + clusters(groups * n.columns * n.mod_splits), splits, st, a, n);
}

}  // namespace slra
