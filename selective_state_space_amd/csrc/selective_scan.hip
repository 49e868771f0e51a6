// The per-channel selective scan: every channel c has its own decay rates
// A[c][n], and with d = softplus(dt + bias_c)
//
//     h[n] <- exp(d A[c][n]) h[n] + d x B[n];   y = sum_n h[n] C[n] + D_c x,
//
// optionally y <- y silu(z).  ("mamba-metal: running Mamba on Apple Silicon",
// the selective scan with a diagonal A per state element.)  The decay differs
// for every (channel, state), so unlike the scalar-decay scan no part of it is
// a matrix product: each state element costs an exponential (two issue
// slots) and four vector operations per token, and forming d, the gate and the
// sums over n some 3 more.  Vector issue is the largest part of the time: 8 x 4096
// tokens of 5120 channels, N 16, take 1.61 million cycles (700 us at 2.3 GHz, 1.9
// TB/s), where the updates alone issue for 0.86 million (20.9 cycles per 64 states,
// the rate of that mix with 4 wavefronts per SIMD) and the other instructions, at
// 2.7 cycles each, for 0.36.  1 x 65536 of 2048 take 840 us in two passes.
//
// A sequence is walked in order, tile by tile (see selective_scan.h for the
// split over lanes).  Where sequences and channels alone do not fill the chip
// the tokens are cut into segments as well: a first pass forms each segment's
// end state from zero and its sum of d, a short one chains them (the decay of
// a whole segment is exp(A sum d)), and the scan then starts every segment
// from its true state.

#include "selective_scan.h"

namespace ssd {

namespace {

// seg [Bt][nseg][Dm][N]: end states from zero (all but the last) become the
// states entering each segment.
__global__ __launch_bounds__(256) void sel_chain_kernel(float *__restrict__ seg,
                                                        const float *__restrict__ dsum,
                                                        const float *__restrict__ A,
                                                        const float *__restrict__ init,
                                                        int64_t total, int32_t Dm, int32_t N,
                                                        int32_t nseg) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;   // (b, c, n)
    if (i >= total) return;
    const int64_t per = (int64_t)Dm * N;
    const int64_t b = i / per, cn = i % per;
    const int64_t c = cn / N;
    const float a2 = rate2(A[cn]);
    float h = init ? init[i] : 0.f;
    float *p = seg + b * nseg * per + cn;
    const float *q = dsum + b * nseg * Dm + c;
    // 8 segments' values in flight at a time (the last end state is not there)
    for (int32_t k0 = 0; k0 < nseg; k0 += 8) {
        float e[8], d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int32_t k = k0 + j;
            e[j] = k + 1 < nseg ? p[k * per] : 0.f;
            d[j] = k + 1 < nseg ? q[(int64_t)k * Dm] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (k0 + j < nseg) p[(k0 + j) * per] = h;
            h = fmaf(fast_exp2(d[j] * a2), h, e[j]);
        }
    }
}

// One token per sequence: the state is read and written once, which is all
// the traffic that counts (A, as large as one sequence's state, comes from L2).
// A lane holds 4 states of R channels; a wavefront's are contiguous, R KB of one
// state (256 sequences, 5120 channels, N 16: 35 us with R 2, 5.1 TB/s; 37 with 4
// channels, or with one channel of 4 sequences).
template <int N, typename Tio, typename Ty, bool GATE, int R>
__global__ __launch_bounds__(256) void sel_step_kernel(
    float *__restrict__ state, const int32_t *__restrict__ slots, int64_t nslots,
    const Tio *__restrict__ x, const Tio *__restrict__ dt, const float *__restrict__ A,
    const Tio *__restrict__ B, const Tio *__restrict__ C, const float *__restrict__ D,
    const Tio *__restrict__ z, const float *__restrict__ dt_bias, Ty *__restrict__ y, int32_t Dm,
    int32_t ncb, int32_t softplus) {
    constexpr int S = SelSplit<N>::S, CPW = SelSplit<N>::CPW, CB = SelSplit<N>::CB;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t cb = blockIdx.x % (uint32_t)ncb;
    const int64_t b = blockIdx.x / (uint32_t)ncb;
    const int s = lane % S;
    const int32_t c0 = (cb * R) * CB + wave * (CPW * R) + lane / S;
    const int64_t slot = slots ? (int64_t)slots[b] : b;
    const bool live = slot >= 0 && slot < nslots;
    float *hp = state + (slot * Dm + c0) * N + 4 * s;
    float4 hv[R], av[R], bv, cv;
    float xv[R], dv[R], zv[R], bias[R], Dc[R];
    if (live) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int32_t c = c0 + r * CPW;
            if (c < Dm) {
                hv[r] = load_nt(hp + (int64_t)r * CPW * N);
                av[r] = *reinterpret_cast<const float4 *>(A + (int64_t)c * N + 4 * s);
                xv[r] = load1(x + b * Dm + c);
                dv[r] = load1(dt + b * Dm + c);
                if constexpr (GATE) zv[r] = load1(z + b * Dm + c);
                bias[r] = dt_bias ? dt_bias[c] : 0.f;
                Dc[r] = D[c];
            }
        }
        bv = widen4(load_raw<false>(B + b * N + 4 * s, 4));
        cv = widen4(load_raw<false>(C + b * N + 4 * s, 4));
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int32_t c = c0 + r * CPW;
        if (c >= Dm) break;
        float out = 0.f;
        if (live) {
            float d = dv[r] + bias[r];
            if (softplus) d = softplus_f(d);
            // (finite up to the largest d: no decay, A = 0, takes 0 d2)
            const float d2 = __builtin_elementwise_minimum(d * kLog2e, 0x1.fffffep127f);
            const float u = d * xv[r];
            float4 h = hv[r];
            h.x = fmaf(fast_exp2(d2 * av[r].x), h.x, u * bv.x);
            h.y = fmaf(fast_exp2(d2 * av[r].y), h.y, u * bv.y);
            h.z = fmaf(fast_exp2(d2 * av[r].z), h.z, u * bv.z);
            h.w = fmaf(fast_exp2(d2 * av[r].w), h.w, u * bv.w);
            store_nt(hp + (int64_t)r * CPW * N, h);
            out = chan_sum<S>(h.x * cv.x + h.y * cv.y + h.z * cv.z + h.w * cv.w);
            out += Dc[r] * xv[r];
            if constexpr (GATE) out *= fast_silu(zv[r]);
        }
        if (s == 0) {
            if constexpr (sizeof(Ty) == 2)
                y[b * Dm + c] = (uint16_t)f32_to_bf16_bits(out);
            else
                y[b * Dm + c] = out;
        }
    }
}

// How a launch is cut: states per lane, and segments of a sequence.
//   * Sequences and channels alone fill the chip (400 workgroups or more with 2
//     states per lane): one segment, as a second pass over the tokens costs
//     more than idle lanes.  2 states per lane give twice the wavefronts of 4
//     (8 x 4096 tokens, 5120 channels, N 16: 705 us against 890, 5 wavefronts
//     per SIMD against 2.5), but 4 do less work per state once they fill it too
//     (16 x 2048 tokens: 682 us against 759).
//   * Else segments of at least 64 tokens, enough for 2048 workgroups of the
//     4-state form (1 x 4096 tokens, 5120 channels: 144 us in 32 segments, 282
//     us in one).  Three launches and a second pass pay from about 256 tokens on:
//     one sequence of 2048 channels, N 16, cut and whole, 128 tokens 14.8 us and
//     11.0, 192 15.0 and 15.6, 256 15.4 and 19.8, 512 18.6 and 37.0; of 5120, 128
//     16.2 and 11.3, 256 20.4 and 19.9, 512 28.8 and 37.9; N 64, 2048 channels, 128
//     20.5 and 18.1, 256 24.1 and 33.6.
struct Cut {
    int ks;
    int64_t ncb, n, len;
};
Cut cut_of(const SelArgs &a) {
    const int64_t few = a.N == 64 ? 4 : 2;   // (16 lanes of a channel at most)
    const int64_t b4 = a.Bt * chan_blocks(a, 4), bf = a.Bt * chan_blocks(a, few);
    Cut s;
    s.ks = (int)(b4 >= 1024 ? 4 : few);
    s.n = 1;
    if (bf > 0 && bf < 400) {
        int64_t n = cdiv64(2048, b4);
        n = n < a.T / 64 ? n : a.T / 64;
        if (n > 1) {
            s.n = n;
            s.ks = (int)(b4 * n >= 1024 ? 4 : few);
        }
    }
    s.ncb = chan_blocks(a, s.ks);
    const int64_t tile = 4 * a.N / s.ks;
    s.len = cdiv64(cdiv64(a.T > 0 ? a.T : 1, s.n), tile) * tile;
    if (s.n > 1) s.n = cdiv64(a.T, s.len);
    return s;
}
size_t seg_bytes(const SelArgs &a, const Cut &s) {
    return s.n > 1 ? (size_t)(a.Bt * s.n * a.Dm * a.N) * sizeof(float) : 0;
}
// f(integral_constant<KS>): the sums over a channel's lanes are built for up to 16
template <int N, typename F>
void by_ks(const Cut &s, F f) {
    if constexpr (N < 64)
        if (s.ks == 2) return f(std::integral_constant<int, 2>());
    f(std::integral_constant<int, 4>());
}

// f(y type): bf16 where the caller asked for the io dtype and that is bf16
template <typename F>
void by_y(const SelArgs &a, F f) {
    if (a.ybf)
        f(uint16_t());
    else
        f(float());
}

}  // namespace

bool selective_scan_fits(const SelArgs &a) {
    if (a.Bt == 0) return true;
    if ((double)a.Bt * (double)chan_blocks(a, 2) > (double)kMaxBlocks) return false;
    const Cut s = cut_of(a);
    return (double)a.Bt * (double)s.n * (double)s.ncb <= (double)kMaxBlocks &&
           (double)a.Bt * (double)a.Dm * (double)a.N <= 256.0 * (double)kMaxBlocks;
}

bool selective_step_fits(const SelArgs &a) {
    return (double)a.Bt * (double)chan_blocks(a) <= (double)kMaxBlocks;
}

size_t selective_scan_workspace(const SelArgs &a) {
    const Cut s = cut_of(a);
    const size_t b = seg_bytes(a, s);
    return b ? b + (size_t)(a.Bt * s.n * a.Dm) * sizeof(float) : 0;
}

SelLayout selective_scan_layout(const SelArgs &a) {
    const Cut s = cut_of(a);
    return SelLayout{s.ks, s.n};
}

// 2 channels per lane where that leaves 2 workgroups per CU
int selective_step_channels(const SelArgs &a) { return a.Bt * chan_blocks(a) >= 2 * 512 ? 2 : 1; }

hipError_t launch_selective_scan(const SelArgs &a, hipStream_t st) {
    const Cut sg = cut_of(a);
    SelGeom g;
    g.T = a.T;
    g.Bt = a.Bt;
    g.Dm = (int32_t)a.Dm;
    g.ncb = (int32_t)sg.ncb;
    g.nseg = (int32_t)sg.n;
    g.seg_len = sg.len;
    g.softplus = a.softplus ? 1 : 0;
    const bool rag = a.Dm % 4 != 0;
    const float *start = a.init;
    hipError_t e = hipSuccess;
    if (sg.n > 1) {
        float *seg = static_cast<float *>(a.ws);
        float *dsum = seg + (size_t)(a.Bt * sg.n * a.Dm * a.N);
        by_state(a, [&](auto n, auto io) {
            typedef decltype(io) Tio;
            by_ks<decltype(n)::value>(sg, [&](auto ks) {
                by_flag(rag, [&](auto r) {
                    sel_scan_kernel<decltype(n)::value, decltype(ks)::value, Tio, float, false,
                                    decltype(r)::value, SCAN_END>
                        <<<dim3((uint32_t)(a.Bt * (sg.n - 1) * g.ncb)), 256, 0, st>>>(
                            (const Tio *)a.x, (const Tio *)a.dt, a.A, (const Tio *)a.B, nullptr,
                            nullptr, nullptr, a.dt_bias, nullptr, a.lens, nullptr, seg, dsum,
                            nullptr, nullptr, g);
                });
            });
        });
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        const int64_t total = a.Bt * a.Dm * a.N;
        sel_chain_kernel<<<dim3((uint32_t)cdiv64(total, 256)), 256, 0, st>>>(
            seg, dsum, a.A, a.init, total, (int32_t)a.Dm, (int32_t)a.N, (int32_t)sg.n);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        start = seg;
    }
    by_state(a, [&](auto n, auto io) {
        typedef decltype(io) Tio;
        by_ks<decltype(n)::value>(sg, [&](auto ks) {
            by_flag(rag, [&](auto r) {
                by_flag(a.z != nullptr, [&](auto gate) {
                    by_y(a, [&](auto yt) {
                        typedef decltype(yt) Ty;
                        if constexpr (sizeof(Ty) == 4 || sizeof(Tio) == 2)   // bf16 y: bf16 io
                            sel_scan_kernel<decltype(n)::value, decltype(ks)::value, Tio, Ty,
                                            decltype(gate)::value, decltype(r)::value, SCAN_OUT>
                                <<<dim3((uint32_t)(a.Bt * sg.n * g.ncb)), 256, 0, st>>>(
                                    (const Tio *)a.x, (const Tio *)a.dt, a.A, (const Tio *)a.B,
                                    (const Tio *)a.C, a.D, (const Tio *)a.z, a.dt_bias, start,
                                    a.lens, (Ty *)a.y, a.fin, nullptr, nullptr, nullptr, g);
                    });
                });
            });
        });
    });
    return hipGetLastError();
}

hipError_t launch_selective_step(const SelArgs &a, hipStream_t st) {
    const int64_t one = chan_blocks(a);
    const bool two = selective_step_channels(a) == 2;
    const int64_t ncb = two ? cdiv64(one, 2) : one;
    const dim3 grid((uint32_t)(ncb * a.Bt));
    by_state(a, [&](auto n, auto io) {
        typedef decltype(io) Tio;
        by_flag(a.z != nullptr, [&](auto gate) {
            by_flag(two, [&](auto f) {
                by_y(a, [&](auto yt) {
                    typedef decltype(yt) Ty;
                    if constexpr (sizeof(Ty) == 4 || sizeof(Tio) == 2)
                        sel_step_kernel<decltype(n)::value, Tio, Ty, decltype(gate)::value,
                                        decltype(f)::value ? 2 : 1><<<grid, 256, 0, st>>>(
                            a.state, a.slots, a.nslots, (const Tio *)a.x, (const Tio *)a.dt, a.A,
                            (const Tio *)a.B, (const Tio *)a.C, a.D, (const Tio *)a.z, a.dt_bias,
                            (Ty *)a.y, (int32_t)a.Dm, (int32_t)ncb, a.softplus ? 1 : 0);
                });
            });
        });
    });
    return hipGetLastError();
}

}  // namespace ssd
