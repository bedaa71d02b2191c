// Gradients of the gated delta rule in chunks of 64 tokens, the chain from a sequence's last chunk to its first.  With dS'
// the gradient of the state behind the chunk, P' and T' transposed,
//
//     g = P' dO + e^(G_end - G) K dS',   x = T' g (the gradient of N),   dv = beta x
//     dS = e^G_end dS' + (scale e^G dO)^T q - (beta e^G x)^T K
//
// As in the forward, transposed, dS' (16 columns x keys) is the left operand of one warp, whose products stay in registers
// from one dS to the next; the other warp of the group adds what does not wait for them: dO' P, the remainders' share of
// dS' K', (scale e^G dO)' q, and the outputs.  What dq and dk need goes to memory rounded to 16 bits (delta_grads.cu); the
// gradients of gates and strengths, which are fp32, come from sums over a row's columns alone:
//
//     dbeta = x.Y,   dg_t = sum over i >= t of (o_i.dO_i - dv_i.v_i) + <S, dS> at the end of the sum
//
// (scaling a token's S by a factor scales every later o but not what a token adds), where the sums run to the end of a group
// of two chunks, whose state the forward has kept in fp32, and dS is the sum of the two terms that the products have of it.
// (The longer the sums, the more of a row's rounding is left in dg: 5.8e-6 of it at 4 x 2048 tokens of 8 heads; groups of four
// and eight chunks 6.5e-6 and 8.4e-6 in 2 to 4 % less time, one chunk 3 to 6 % more.  Where a head keeps little of its
// state from token to token the sums cancel most: there groups of two leave 8e-6, of eight 1.4e-5.)
//
// 3.8 us a chunk of 32 columns (4 x 2048 tokens of 8 heads 123 us), bound by the second warp's 232 products and its outputs.
// Both roles share one count of registers, 255, and keys of 128 spill 180 to 192 bytes (bf16; the forward's chain 20).
#include "delta_chain.cuh"

namespace gla {
namespace {

template <typename T, int KD, int VG>
__global__ void __launch_bounds__(64 * VG, 1) delta_chain_back_kernel(const __grid_constant__ ChainMaps maps, DeltaArgs a, int tiles)
{
    typedef ChainShared<KD, VG, 2, DeltaCellRows> Shared;
    constexpr int kThreads = 64 * VG;
    extern __shared__ __align__(1024) char raw[];
    Shared &sh = *reinterpret_cast<Shared *>(raw);
    ChainWalk w;
    bars_init(sh.full);
    tc::grid_dep_wait();
    if (!chain_walk(a, tiles, 16 * VG, w))
        return;
    const int tid = threadIdx.x, lane = tid % 32, group = tid / 32 % VG;
    const bool output = tid >= kThreads / 2;
    const int col = w.v0 + 16 * group + lane / 4, two = 2 * (lane % 4);
    const bool on = w.v0 + 16 * group < a.V;
    const size_t state = (w.head * a.K + two) * a.V;
    const DeltaTrace trace = a.trace;
    const int g16 = (w.v0 >> 4) + group;

    Power in[2] = {{1.f, 1.f}, {1.f, 1.f}};   // fp16: the powers of the columns of dS
    auto chain = [&](typename Shared::Stage &st, float (&s)[KD / 8][4]) {
        const float4 *row = st.cell.row;
        float x[8][4] = {};
        {
            uint32_t s_hi[KD / 16][4];
            if constexpr (kScaled<T>)
                if (lane % 4 == 0) {
                    sh.power[group][lane / 4] = in[0].from;
                    sh.power[group][lane / 4 + 8] = in[1].from;
                }
#pragma unroll
            for (int i = 0; i < KD / 16; ++i) {
                uint32_t s_lo[4];
                split_rows<T>(s[2 * i], s[2 * i + 1], in, s_hi[i], s_lo);
                sh.state[group][i][0][lane] = as_uint4(s_hi[i]);
                sh.state[group][i][1][lane] = as_uint4(s_lo);
            }
            bar_tell(kBarState + group);
            state_by_rows<T, KD, false>(x, s_hi, s_hi, st.k, lane);
        }
        const float last = row[kDeltaChunk - 1].y;
#pragma unroll
        for (int j = 0; j < KD / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[j][e] *= last;
        bar_sync(kBarShare + group);
        // of products with a column of dS that was divided by its power
        auto of = [](float f, const Power &p) { return kScaled<T> ? f * p.from : f; };
        Power by[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // g, and x = g + (T' - I) g
            uint32_t hi[4];
            float r[2][4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int j = 2 * i + y;
                const float4 p = sh.ks[group][j][lane];
                const float f0 = row[8 * j + two].z, f1 = row[8 * j + two + 1].z;
                r[y][0] = fmaf(of(f0, in[0]), x[j][0], p.x), r[y][1] = fmaf(of(f1, in[0]), x[j][1], p.y);
                r[y][2] = fmaf(of(f0, in[1]), x[j][2], p.z), r[y][3] = fmaf(of(f1, in[1]), x[j][3], p.w);
                x[j][0] = r[y][0], x[j][1] = r[y][1], x[j][2] = r[y][2], x[j][3] = r[y][3];
            }
            if constexpr (!kScaled<T>)
                triangle_step<T, true, 2>(x, r[0], r[1], hi, i, st.cell.inverse, lane);
        }
        if constexpr (kScaled<T>)
            triangle_rows<T, true, 2>(x, st.cell.inverse, lane);
        uint32_t hi[4][4], lo[4][4];
        auto update = [&](float (&u)[4], int j) {
            const float4 c0 = row[8 * j + two], c1 = row[8 * j + two + 1];
            const float f0 = -c0.x * c0.y, f1 = -c1.x * c1.y;
            u[0] = f0 * x[j][0], u[1] = f1 * x[j][1], u[2] = f0 * x[j][2], u[3] = f1 * x[j][3];
        };
        if constexpr (kScaled<T>) {   // they are added to dS: one power for both
            float most[2] = {};
            rows_largest(s, most);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float u[1][4];
                update(u[0], j);
                rows_largest(u, most);
            }
            rows_power<kState>(most, by);
#pragma unroll
            for (int j = 0; j < KD / 8; ++j)
                times_rows(s[j], s[j], by[0].to, by[1].to);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float u[2][4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int j = 2 * i + y;
                sh.n[group][j][lane] = as_float4(x[j]);
                update(u[y], j);
            }
            split_rows<T>(u[0], u[1], by, hi[i], lo[i]);
        }
        bar_tell(kBarRows + group);
        state_add<T, KD>(s, hi, lo, st.k, lane);
        bar_sync(kBarShare + group);   // the other warp's part of dS
        const float4 *part = reinterpret_cast<const float4 *>(sh.state[group]) + lane;
#pragma unroll
        for (int j = 0; j < KD / 8; ++j) {
            const float4 p = part[j * 32];
            if constexpr (kScaled<T>) {
                s[j][0] = fmaf(by[0].from, s[j][0], p.x), s[j][1] = fmaf(by[0].from, s[j][1], p.y);
                s[j][2] = fmaf(by[1].from, s[j][2], p.z), s[j][3] = fmaf(by[1].from, s[j][3], p.w);
            } else {
                s[j][0] += p.x, s[j][1] += p.y, s[j][2] += p.z, s[j][3] += p.w;
            }
        }
        if constexpr (kScaled<T>)
            rows_power<kState>(s, in);
    };
    constexpr bool kChecked = std::is_same_v<T, __half>;
    bool bad = false;
    auto help = [&](typename Shared::Stage &st, int c) {
        const float4 *row = st.cell.row;
        const size_t cell = (size_t)(w.slot + c) * a.HV + w.hv;
        const float score = kScaled<T> ? a.score[cell] : 1.f;   // P's factor
        float in_from[2] = {1.f, 1.f};
        uint32_t d_hi[4][4], d_lo[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            values_t<VG>(d_hi[i], st.v[1], i, group, lane);
        float g[8][4] = {};
#pragma unroll
        for (int i = 3; i >= 0; --i)
#pragma unroll
            for (int j = 0; j <= 2 * i + 1; ++j) {
                const uint4 b = st.cell.score[triangle_at_t(j, i) * 32 + lane];
                mma<T>(g[j], d_hi[i], b.x, b.y);
                mma<T>(g[j], d_hi[i], b.z, b.w);
            }
        bar_sync(kBarState + group);
        {
            uint32_t s_in[KD / 16][4];
            float k[8][4] = {};
            if constexpr (kScaled<T>) {
                in_from[0] = sh.power[group][lane / 4], in_from[1] = sh.power[group][lane / 4 + 8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    times_rows(g[j], g[j], score, score);
            }
#pragma unroll
            for (int i = 0; i < KD / 16; ++i)
                take(s_in[i], sh.state[group][i][1][lane]);
            state_by_rows<T, KD, false>(k, s_in, s_in, st.k, lane);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float f0 = row[8 * j + two].z, f1 = row[8 * j + two + 1].z;
                if constexpr (kScaled<T>)
                    times_rows(k[j], k[j], in_from[0], in_from[1]);
                sh.ks[group][j][lane] = make_float4(fmaf(f0, k[j][0], g[j][0]), fmaf(f1, k[j][1], g[j][1]), fmaf(f0, k[j][2], g[j][2]),
                                                    fmaf(f1, k[j][3], g[j][3]));
            }
            bar_tell(kBarShare + group);
#pragma unroll
            for (int i = 0; i < KD / 16; ++i)
                take(s_in[i], sh.state[group][i][0][lane]);
            if constexpr (kScaled<T>) {
                const float most = group_largest(in_from);
                to_group<KD / 16>(s_in, in_from, most);
                if (on && lane == 0)
                    trace.power[(cell * (a.V / 16) + g16) * 8 + 4] = most;
            }
            if (on)
                put_blocks<KD / 16>(trace.ds + cell * trace.s_size, s_in, 2 * g16, KD / 8, lane);
        }
        {   // (scale e^G dO)' q, to where the state's rounded values lay
            auto started = [&](float (&r)[2][4], int i) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float f0 = row[16 * i + 8 * e + two].w, f1 = row[16 * i + 8 * e + two + 1].w;
                    const float2 d0 = widen2<T>(d_hi[i][2 * e]), d1 = widen2<T>(d_hi[i][2 * e + 1]);
                    r[e][0] = f0 * d0.x, r[e][1] = f1 * d0.y, r[e][2] = f0 * d1.x, r[e][3] = f1 * d1.y;
                }
            };
            Power by[2];
            if constexpr (kScaled<T>) {
                float most[2] = {};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float r[2][4];
                    started(r, i);
                    rows_largest(r, most);
                }
                rows_power<kOperand>(most, by);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float r[2][4];
                started(r, i);
                split_rows<T>(r[0], r[1], by, d_hi[i], d_lo[i]);
            }
            float s[KD / 8][4] = {};
            state_add<T, KD>(s, d_hi, d_lo, st.q, lane);
            if constexpr (kScaled<T>)
#pragma unroll
                for (int j = 0; j < KD / 8; ++j)
                    times_rows(s[j], s[j], by[0].from, by[1].from);
            float4 *part = reinterpret_cast<float4 *>(sh.state[group]) + lane;
            __syncwarp();   // all lanes have the rounded values
#pragma unroll
            for (int j = 0; j < KD / 8; ++j)
                part[j * 32] = as_float4(s[j]);
        }
        float4 y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] = on ? trace.y[(cell * (a.V / 16) + g16) * 256 + j * 32 + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
        bar_sync(kBarRows + group);
        bar_tell(kBarShare + group);
        const int rows = min(kDeltaChunk, w.len - c * kDeltaChunk);
        T *dv = static_cast<T *>(a.dv) + (((size_t)w.bos + (size_t)c * kDeltaChunk) * a.HV + w.hv) * a.V + col;
        float sum[32];   // x.Y, then dv.v
        Power to_x = {1.f, 1.f};
        if constexpr (kScaled<T>) {   // beta x goes to the gradients of k, as a group's columns have one power
            float most = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float4 x = sh.n[group][j][lane];
                const float b0 = row[8 * j + two].x, b1 = row[8 * j + two + 1].x;
                most = fmaxf(most, fmaxf(fmaxf(fabsf(b0 * x.x), fabsf(b1 * x.y)), fmaxf(fabsf(b0 * x.z), fabsf(b1 * x.w))));
            }
            to_x = power_of<kTerm>(warp_largest(most));
            if (on && lane == 0)
                trace.power[(cell * (a.V / 16) + g16) * 8 + 5] = to_x.from;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t v[4], xw[4];
            values_t<VG>(v, st.v[0], i, group, lane);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = 2 * i + e, t = 8 * j + two;
                const float4 x = sh.n[group][j][lane];
                const float b0 = row[t].x, b1 = row[t + 1].x;
                if constexpr (kChecked)
                    bad |= lost(x.x) || lost(x.y) || lost(x.z) || lost(x.w);
                const float2 v0 = widen2<T>(v[2 * e]), v1 = widen2<T>(v[2 * e + 1]);
                const float r0 = kScaled<T> ? b0 * to_x.to : 1.f, r1 = kScaled<T> ? b1 * to_x.to : 1.f;
                xw[2 * e] = narrow2<T>(make_float2(r0 * x.x, r1 * x.y));
                xw[2 * e + 1] = narrow2<T>(make_float2(r0 * x.z, r1 * x.w));
                sum[2 * j] = fmaf(x.x, y[j].x, x.z * y[j].z);
                sum[2 * j + 1] = fmaf(x.y, y[j].y, x.w * y[j].w);
                sum[16 + 2 * j] = b0 * fmaf(x.x, v0.x, x.z * v1.x);
                sum[17 + 2 * j] = b1 * fmaf(x.y, v0.y, x.w * v1.y);
                if (on && t < rows) {
                    dv[(size_t)t * a.HV * a.V] = narrow<T>(b0 * x.x);
                    dv[(size_t)t * a.HV * a.V + 8] = narrow<T>(b0 * x.z);
                }
                if (on && t + 1 < rows) {
                    dv[(size_t)(t + 1) * a.HV * a.V] = narrow<T>(b1 * x.y);
                    dv[(size_t)(t + 1) * a.HV * a.V + 8] = narrow<T>(b1 * x.w);
                }
            }
            if (on) {
                const uint32_t one[1][4] = {{xw[0], xw[1], xw[2], xw[3]}};
                put_blocks<1>(trace.x + cell * trace.n_size + 2 * i * 32, one, 2 * g16, 8, lane);
            }
        }
        sum_over_columns<32>(sum, lane);   // lane / 4 is left with two tiles of one of the two
        if (on) {
            float *to = trace.dots + ((cell * (a.V / 16) + g16) * 3 + 1 + lane / 16) * 64 + 16 * (lane / 4 % 4) + two;
            *reinterpret_cast<float2 *>(to) = make_float2(sum[0], sum[1]);
            *reinterpret_cast<float2 *>(to + 8) = make_float2(sum[2], sum[3]);
        }
    };

    constexpr size_t kCell = sizeof(DeltaCellBack);
    auto walk = [&](auto work) {
        if (tid == kThreads / 2 && w.chunks)
            ask_chunk(a, maps, w, sh, w.chunks - 1, 0, kCell, kCellRows);
        for (int turn = 0; turn < w.chunks; ++turn) {
            const int c = w.chunks - 1 - turn;
            const bool ok = tc::bar_wait(&sh.full[turn & 1], (turn >> 1) & 1);
            if (__syncthreads_or(!ok)) {
                give_up(a.status, &sh.full[turn & 1], (turn >> 1) & 1);
                return;
            }
            if (tid == kThreads / 2 && c > 0)
                ask_chunk(a, maps, w, sh, c - 1, turn + 1, kCell, kCellRows);
            if (w.len - c * kDeltaChunk < kDeltaChunk) {
                clear_tail<VG>(sh.stage[turn & 1], w.len - c * kDeltaChunk);
                __syncthreads();
            }
            work(sh.stage[turn & 1], c);
        }
    };
    if (!output) {
        float s[KD / 8][4];
        state_io<KD>(s, nullptr, a.dht, state, a.V, col, on, false);
        auto across = [&](int c) {   // <S, dS> behind chunk c, of the dS that the products have
            const size_t at = delta_kept_at(a, w.n, c, w.hv, g16);
            const float4 *kept = trace.kept + at * (KD / 8 * 32) + lane;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < KD / 8; ++j) {
                const float4 p = kept[j * 32];
                const float2 d0 = in_two<T>(s[j][0], s[j][1], in[0]), d1 = in_two<T>(s[j][2], s[j][3], in[1]);
                sum += (p.x * d0.x + p.y * d0.y) + (p.z * d1.x + p.w * d1.y);
            }
#pragma unroll
            for (int m = 16; m; m /= 2)
                sum += __shfl_xor_sync(~0u, sum, m);
            if (lane == 0)
                trace.across[at] = sum;
        };
        if constexpr (kScaled<T>)
            rows_power<kState>(s, in);
        if (on && w.chunks)
            across(w.chunks - 1);
        walk([&](auto &st, int c) {
            chain(st, s);
            if (on && c > 0 && c % kDeltaKept == 0)   // while the other warp is at its outputs
                across(c - 1);
        });
        report_lost<T>(a, s, false);
        if (a.dh0)
            state_io<KD>(s, a.dh0, nullptr, state, a.V, col, on, true);
    } else {
        walk([&](auto &st, int c) { help(st, c); });
        if (kChecked && bad)
            report(a.status, GLA_ERR_RANGE);
    }
}

// dg and dbeta of a group of chunks, a thread a row: sums over the head's columns, then from the group's last row on.
__global__ void __launch_bounds__(kDeltaChunk *kDeltaKept) delta_chunk_gates_kernel(DeltaArgs a)
{
    constexpr int kRows = kDeltaChunk * kDeltaKept;
    __shared__ float part[kRows / 32];
    tc::grid_dep_wait();
    const int group = blockIdx.x / a.HV, hv = blockIdx.x - group * a.HV, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    int lo = 0, hi = a.N - 1;   // the last sequence whose groups start at or before this one
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (delta_first_group(a, mid) <= group)
            lo = mid;
        else
            hi = mid - 1;
    }
    int bos, len;
    if (!delta_sequence(a, lo, bos, len))
        return;
    const int first = group - delta_first_group(a, lo), t = first * kRows + tid, groups = a.V / 16;
    if (first < 0 || (int64_t)first * kRows >= len)
        return;
    float dG = 0.f, end = 0.f;
    if (t < len) {
        const size_t cell = (size_t)(delta_first_slot(a, lo) + t / kDeltaChunk) * a.HV + hv;
        const float *dots = a.trace.dots + cell * groups * 192 + t % kDeltaChunk;
        float beta = 0.f;
        for (int g = 0; g < groups; ++g) {
            dG += dots[g * 192] - dots[g * 192 + 128];
            beta += dots[g * 192 + 64];
        }
        a.dbeta[(size_t)(bos + t) * a.HV + hv] = beta;
    }
    for (int g = 0; g < groups; ++g)
        end += a.trace.across[((size_t)group * a.HV + hv) * groups + g];
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
        const float u = __shfl_down_sync(~0u, dG, m);
        if (lane + m < 32)
            dG += u;
    }
    if (lane == 0)
        part[warp] = dG;
    __syncthreads();
    float behind = 0.f;
    for (int i = kRows / 32 - 1; i > warp; --i)
        behind += part[i];
    if (t < len)
        a.dg[(size_t)(bos + t) * a.HV + hv] = dG + (behind + end);
}

}  // namespace

cudaError_t launch_delta_chain_back(const DeltaArgs &a, bool half, cudaStream_t s)
{
    auto go = [&](auto t, auto kd, auto vg) {
        typedef std::remove_pointer_t<decltype(t)> T;
        constexpr int KD = decltype(kd)::value, VG = decltype(vg)::value;
        return launch_chain(delta_chain_back_kernel<T, KD, VG>, sizeof(ChainShared<KD, VG, 2, DeltaCellRows>), VG, half, a, s);
    };
    auto by_keys = [&](auto t, auto vg) { return a.K == 128 ? go(t, Int<128>(), vg) : go(t, Int<64>(), vg); };
    auto by_type = [&](auto vg) { return half ? by_keys((__half *)0, vg) : by_keys((__nv_bfloat16 *)0, vg); };
    return few_columns(a) ? by_type(Int<2>()) : by_type(Int<4>());
}

cudaError_t launch_delta_chunk_gates(const DeltaArgs &a, cudaStream_t s)
{
    constexpr int kRows = kDeltaChunk * kDeltaKept;
    const int groups = a.cu ? a.T / kRows + a.N : a.B * ((a.T + kRows - 1) / kRows);
    return launch_early(delta_chunk_gates_kernel, (unsigned)((size_t)groups * a.HV), kRows, s, a);
}

}  // namespace gla
