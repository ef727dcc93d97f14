// Helpers of the row kernels (residual_norm.cuh, qk_rope.cuh): typed vectors of eight elements, each
// thread's own ring of asynchronous loads, and sums over the threads that share a row.
//
// These kernels move few bytes per element and are bound by memory only while they issue few enough
// instructions: an SM has about 22 bytes of HBM bandwidth a clock, so a vector of eight bf16 elements read
// and written leaves its warp some 180 issue slots.  Hence the packed fp32 arithmetic (two lanes of a
// register pair an instruction), the sums that halve the values they carry at each exchange, and loops that
// keep the bookkeeping of samples out of their rows (all three: 5120 channels forward 892 -> 481 us).
#pragma once

#include "common.cuh"

namespace slra {

// Element types of the tensors, as the values of slra_dtype.
constexpr int kBf16 = 0, kF32 = 1, kF16 = 2;

// Packed fp32 arithmetic: two independent IEEE operations.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
          "l"(reinterpret_cast<unsigned long long&>(c)));
    return reinterpret_cast<float2&>(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return reinterpret_cast<float2&>(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return reinterpret_cast<float2&>(d);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float fold(float2 a) { return a.x + a.y; }

// Eight elements of a row, in fp32.
struct Vec {
    float2 f[4];
};
__device__ __forceinline__ Vec vec_of(float x) {
    Vec v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v.f[i] = both(x);
    return v;
}

// In memory: one 16-byte unit of a 16-bit type, two of fp32.
template <typename T>
constexpr int kUnits = sizeof(T) / 2;

template <typename T>
__device__ __forceinline__ Vec unpack(const uint4 (&u)[kUnits<T>]);
template <>
__device__ __forceinline__ Vec unpack<__nv_bfloat16>(const uint4 (&u)[1]) {
    const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
    Vec v;
#pragma unroll
    for (int i = 0; i < 4; ++i)  // bf16 is the upper half of fp32
        v.f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    return v;
}
template <>
__device__ __forceinline__ Vec unpack<__half>(const uint4 (&u)[1]) {
    const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
    Vec v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v.f[i] = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    return v;
}
template <>
__device__ __forceinline__ Vec unpack<float>(const uint4 (&u)[2]) {
    Vec v;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        v.f[2 * i] = make_float2(__uint_as_float(u[i].x), __uint_as_float(u[i].y));
        v.f[2 * i + 1] = make_float2(__uint_as_float(u[i].z), __uint_as_float(u[i].w));
    }
    return v;
}

// Rounded to nearest even, once, on the way to memory.
template <typename T>
__device__ __forceinline__ void pack(const Vec& v, uint4 (&u)[kUnits<T>]);
template <>
__device__ __forceinline__ void pack<__nv_bfloat16>(const Vec& v, uint4 (&u)[1]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v.f[i].x, v.f[i].y);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    u[0] = make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ void pack<__half>(const Vec& v, uint4 (&u)[1]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(v.f[i].x, v.f[i].y);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    u[0] = make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ void pack<float>(const Vec& v, uint4 (&u)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
        u[i] = make_uint4(__float_as_uint(v.f[2 * i].x), __float_as_uint(v.f[2 * i].y),
                          __float_as_uint(v.f[2 * i + 1].x), __float_as_uint(v.f[2 * i + 1].y));
}

// A vector's eight elements in memory are consecutive, or (SPLIT) two runs of four, the second `gap`
// elements on.  Split vectors serve rotary pairs of a head's two halves, and rows in fp32: there a warp's
// 16-byte accesses then cover consecutive memory, where eight consecutive elements a thread would touch
// every line twice (1536 channels forward with an fp32 stream: 133 -> 113 us).
template <typename T, bool SPLIT = false>
__device__ __forceinline__ Vec load_vec(const T* p, int gap = 4) {
    uint4 u[kUnits<T>];
    if constexpr (SPLIT && sizeof(T) == 2) {
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(p)), b = __ldg(reinterpret_cast<const uint2*>(p + gap));
        u[0] = make_uint4(a.x, a.y, b.x, b.y);
    } else {
#pragma unroll
        for (int i = 0; i < kUnits<T>; ++i) u[i] = __ldg(reinterpret_cast<const uint4*>(p + i * (SPLIT ? gap : 4)));
    }
    return unpack<T>(u);
}
template <typename T, bool SPLIT = false>
__device__ __forceinline__ void store_vec(T* p, const Vec& v, int gap = 4) {
    uint4 u[kUnits<T>];
    pack<T>(v, u);
    if constexpr (SPLIT && sizeof(T) == 2) {
        *reinterpret_cast<uint2*>(p) = make_uint2(u[0].x, u[0].y);
        *reinterpret_cast<uint2*>(p + gap) = make_uint2(u[0].z, u[0].w);
    } else {
#pragma unroll
        for (int i = 0; i < kUnits<T>; ++i) *reinterpret_cast<uint4*>(p + i * (SPLIT ? gap : 4)) = u[i];
    }
}

// Eight elements of a vector whose type is known at run time (weights, modulation rows), or `fill`
// where there is no such vector.
template <bool SPLIT = false>
__device__ __forceinline__ Vec load_any(const void* base, long long at, int dtype, float fill, int gap = 4) {
    if (!base) return vec_of(fill);
    if (dtype == kF32) return load_vec<float, SPLIT>(static_cast<const float*>(base) + at, gap);
    if (dtype == kBf16) return load_vec<__nv_bfloat16, SPLIT>(static_cast<const __nv_bfloat16*>(base) + at, gap);
    return load_vec<__half, SPLIT>(static_cast<const __half*>(base) + at, gap);
}

// Asynchronous copies global -> shared.  Every thread reads back only what it copied itself, so its own
// wait orders the data and no barrier is needed.
__device__ __forceinline__ void async_copy16(uint32_t smem, const void* gmem) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
}
__device__ __forceinline__ void async_copy8(uint32_t smem, const void* gmem) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem), "l"(gmem) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 shared16(uint32_t smem) {
    uint4 u;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "r"(smem)
                 : "memory");
    return u;
}
__device__ __forceinline__ uint32_t shared_address(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// A thread's own part of a ring of `stages` rows: unit u of the stage at `at` is at + u * unit.  One stage
// is filled (at `in`) while the oldest is read (at `out`).
struct Ring {
    uint32_t in, out, first, last, stage, unit;
    // `units` 16-byte units a thread and stage
    __device__ Ring(uint32_t base, int stages, int units) {
        unit = blockDim.x * 16;
        stage = unit * units;
        first = in = out = base + threadIdx.x * 16;
        last = first + stage * (stages - 1);
    }
    __device__ __forceinline__ void filled() { in = in == last ? first : in + stage; }
    __device__ __forceinline__ void done() { out = out == last ? first : out + stage; }
    template <bool SPLIT = false, typename T>
    __device__ __forceinline__ void copy(int u, const T* p, int gap = 4) const {
        if constexpr (SPLIT && sizeof(T) == 2) {
            async_copy8(in + u * unit, p);
            async_copy8(in + u * unit + 8, p + gap);
        } else {
#pragma unroll
            for (int i = 0; i < kUnits<T>; ++i) async_copy16(in + (u + i) * unit, p + i * (SPLIT ? gap : 4));
        }
    }
    template <typename T>
    __device__ __forceinline__ Vec read(int u) const {
        uint4 w[kUnits<T>];
#pragma unroll
        for (int i = 0; i < kUnits<T>; ++i) w[i] = shared16(out + (u + i) * unit);
        return unpack<T>(w);
    }
    // Units [u, u + n) of every stage, for a vector that is never copied.
    __device__ __forceinline__ void clear(int u, int n) const {
        for (uint32_t s = first;; s += stage) {
            for (int i = 0; i < n; ++i)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(s + (u + i) * unit), "r"(0) : "memory");
            if (s == last) break;
        }
    }
};

// A step's copies are committed `stages` - 1 steps ahead (1 to 4 stages); the oldest have arrived.
__device__ __forceinline__ void ring_wait(int stages) {
    if (stages == 3) async_wait<2>();
    else if (stages == 4) async_wait<3>();
    else if (stages == 2) async_wait<1>();
    else async_wait<0>();
}
constexpr int kMaxStages = 4;

// A worker's rows in order: `each` for a row while there are any, `next` moves pointers on to the following
// one, `wrap` from behind a sample's last token to the next sample.
struct Feed {
    int run, left, tokens;  // rows until the next sample or the end, rows behind them
    __device__ Feed(int n, int l0, int per_sample) : tokens(per_sample) {
        run = min(n, tokens - l0);
        left = n - run;
    }
    template <class Each, class Next, class Wrap>
    __device__ __forceinline__ void row(Each each, Next next, Wrap wrap) {
        if (run > 0) {
            each();
            next();
            if (--run == 0 && left > 0) {
                wrap();
                run = min(left, tokens);
                left -= run;
            }
        }
    }
};

// A team of threads shares a row: the whole block (WIDE; a multiple of 32 threads, at most 1024), or
// `size` threads of a warp, a power of two (then several teams in a block).
constexpr int kTeamSums = 4;                      // values that are summed at once, at most
constexpr int kTeamScratch = 2 * kTeamSums * 32;  // floats of shared memory for a block-wide team's sums

template <bool WIDE>
struct Team {
    int size;
    float* scratch;  // kTeamScratch floats, zero before the first sum (a block-wide team)
    int turn = 0;    // which half of the scratch the next sum uses

    __device__ Team(int n, float* s) : size(n), scratch(s) {
        if (WIDE) {
            for (int i = threadIdx.x; i < kTeamScratch; i += blockDim.x) s[i] = 0.f;
            __syncthreads();
        }
    }
    __device__ __forceinline__ void sync() const {
        if (WIDE) __syncthreads();
        else __syncwarp();
    }
    static __device__ __forceinline__ float swap(float x, int o) { return __shfl_xor_sync(0xffffffffu, x, o); }

    // Every value summed over the team, in a fixed order; each thread gets the sums.  In a warp, lanes that
    // exchange several values keep half of them each time, so that four values cost six shuffles and end
    // in eight lanes each.  Across warps: one write, one barrier, and each lane adds its share of the warps'
    // values.  Consecutive sums use the scratch's halves in turn: before a thread can write a half again,
    // every thread has passed the other half's barrier and so has read this one.
    template <int N>
    __device__ __forceinline__ void sum(float (&v)[N]) {
        static_assert(N == 1 || N == 2 || N == 4, "");
        if (!WIDE) {
            for (int o = size >> 1; o > 0; o >>= 1)
#pragma unroll
                for (int n = 0; n < N; ++n) v[n] += swap(v[n], o);
            return;
        }
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        float k[N];
#pragma unroll
        for (int n = 0; n < N; ++n) k[n] = v[n];
#pragma unroll
        for (int o = 16, left = N; o > 0; o >>= 1) {
            if (left > 1) {  // keep the upper or the lower half of the values
                left >>= 1;
                const bool up = lane & o;
#pragma unroll
                for (int n = 0; n < left; ++n) {
                    const float give = up ? k[n] : k[n + left];
                    k[n] = (up ? k[n + left] : k[n]) + swap(give, o);
                }
            } else {
                k[0] += swap(k[0], o);
            }
        }
        constexpr int span = 32 / N;  // lanes a value
        float* s = scratch + turn * (kTeamSums * 32);
        turn ^= 1;
        if (lane % span == 0) s[lane / span * 32 + warp] = k[0];
        __syncthreads();
        // eight float4 of warps' values a sum
        const float4* f = reinterpret_cast<const float4*>(s) + lane / span * 8;
        const float4 a = f[lane & 7];
        k[0] = (a.x + a.y) + (a.z + a.w);
        k[0] += swap(k[0], 4);
        k[0] += swap(k[0], 2);
        k[0] += swap(k[0], 1);
        const float all = k[0];
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] = N == 1 ? all : __shfl_sync(0xffffffffu, all, n * span);
    }
};

// Where a worker stands in a tensor of rows with free batch and token strides.  The same for all threads of
// a block-wide team, so that it takes none of their registers.
template <typename T>
struct RowWalk {
    char* p;
    long long step, back;  // bytes to the next token, and from behind a sample's last token to the next sample
    // element strides of batch and token; from token l of sample b
    __device__ RowWalk(const void* base, long long sb, long long sl, int b, int l, int tokens)
        : p(const_cast<char*>(static_cast<const char*>(base)) + (b * sb + l * sl) * static_cast<int>(sizeof(T))),
          step(sl * static_cast<int>(sizeof(T))),
          back((sb - tokens * sl) * static_cast<int>(sizeof(T))) {}
    __device__ RowWalk(const RowTensor& t, int b, int l, int tokens) : RowWalk(t.p, t.b, t.l, b, l, tokens) {}
    __device__ __forceinline__ T* at(int c) const {  // element c
        return reinterpret_cast<T*>(p + static_cast<unsigned>(c * static_cast<int>(sizeof(T))));
    }
    __device__ __forceinline__ void next() { p += step; }
    __device__ __forceinline__ void wrap() { p += back; }
};

// Threads of a block for a row of `slots` vectors, with `V` vectors a thread: rows of up to 32 vectors
// share a block of 128 threads.
inline void row_team(int slots, int V, RowPlan* p) {
    p->V = V;
    if (slots <= 32) {
        p->team = 1;
        while (p->team < slots) p->team *= 2;
        p->threads = 128;
    } else {
        p->team = p->threads = ((slots + V - 1) / V + 31) / 32 * 32;
    }
}
// One worker a team, on consecutive rows, as many as the blocks up to `most` make necessary.
inline void row_workers(long long rows, int most, RowPlan* p) {
    const int teams = p->threads / p->team;
    const long long cap = static_cast<long long>(kMaxWorkers / teams < most ? kMaxWorkers / teams : most) * teams;
    p->share = static_cast<int>((rows + cap - 1) / cap);
    const long long workers = (rows + p->share - 1) / p->share;
    p->blocks = static_cast<int>((workers + teams - 1) / teams);
    p->workers = p->blocks * teams;
    p->parts = 1;
}
// Stages of a ring: enough that an SM's blocks keep 96 KB of copies in flight (about twice what its share of
// the bandwidth moves in the time a load takes), within `room` bytes a block, and no more than a worker of
// `most` rows takes steps of `rows`.  `early`: a stage is read at once and filled again before its arithmetic.
inline int ring_stages(size_t stage, int blocks_per_sm, size_t room, long long most, int rows, bool early = false) {
    int n = early ? 1 : 2;
    while (n < kMaxStages && (n - (early ? 0 : 1)) * stage * blocks_per_sm < 96 * 1024) ++n;
    while (n > 1 && (n * stage > room || (n - 1ll) * rows >= most)) --n;
    return n;
}

// Before a launch with `bytes` of dynamic shared memory.  The limit belongs to the function, not to the call: `most`
// is the same in every call of a kernel, or one call could lower it between another host thread's setting and launch.
template <typename K>
cudaError_t allow_shared(K kernel, size_t bytes, size_t most) {
    if (bytes <= 40 * 1024) return cudaSuccess;  // 48 KB without opting in, less the static part
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
}

// The sums of partial sums: kernels of `kFinalWarps` warps a block.  Where a job has many, the blocks of a
// cluster share it.
constexpr int kFinalWarps = 16;

// The joining kernel's blocks start while the row kernel's last ones end, and wait for all it has written.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_rows() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Adds the totals of the cluster's other blocks to warp 0's `sum` in its first block, in the blocks' order.
template <int N>
__device__ __forceinline__ void join_cluster(float (&total)[N][32], float (&sum)[N], int splits) {
    auto barrier = []() {
        asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    };
    __syncwarp();
    barrier();
    if (blockIdx.x % splits == 0 && threadIdx.x < 32)
        for (int z = 1; z < splits; ++z)
#pragma unroll
            for (int n = 0; n < N; ++n) {
                uint32_t at;
                float x;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(shared_address(&total[n][threadIdx.x])), "r"(z));
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
                sum[n] += x;
            }
    barrier();  // the others' memory stays until it is read
}
// Blocks of a cluster for each of `jobs` jobs of up to `most` partial sums: two or more sums for every warp,
// while the blocks start together (four an SM).
inline int join_splits(long long most, long long jobs) {
    int n = 1;
    while (n < 8 && most > 2ll * kFinalWarps * n && 2 * n * jobs <= 4 * kSMs) n *= 2;
    return n;
}
// `blocks`: a multiple of `splits`.
template <typename... P, typename... A>
cudaError_t launch_join(void (*kernel)(P...), long long blocks, int splits, cudaStream_t st, const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(32 * kFinalWarps);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace slra
