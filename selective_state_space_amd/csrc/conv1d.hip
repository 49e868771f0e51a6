// The short causal convolution in front of the scan: per channel c,
//     pre_t = bias_c + sum_k w[c][k] x_{t-(W-1)+k},   y_t = pre_t (or silu(pre_t)),
// with the W-1 tokens before the first taken from a carried state.
//
// Every output needs 2W operations for 2 elements moved, so all three kernels
// are bound by memory.  A lane owns 4 consecutive channels and walks along the
// tokens with the last W-1 inputs in registers: x is read once (plus W-1 rows per
// run of tokens), and each row of a wavefront is 512 bytes (bf16) or 1 KB (float32)
// contiguous.  The times below are those of replayed graphs on one card.
// The outputs go to up to three dense tensors (x, B and C of the scan), so the
// scan needs no copy of a strided slice; a lane's channels never cross from
// one tensor into the next, and a lane whose channels run past a tensor's end
// moves its elements one by one.

#include <type_traits>

#include "layer_launch.h"
#include "ssd_device.h"

namespace ssd {

namespace {

constexpr int kVec = 4;   // channels of a lane

// V consecutive elements as stored.  Rows of an odd width or a slice start at
// any element, so the copies below assume element alignment only (the global
// memory path takes unaligned 8- and 16-byte accesses).  RAG: n may be less than V.
template <typename T, int V>
struct Vec {
    T v[V];
};
template <int BYTES>
struct Words;
template <>
struct Words<8> {
    typedef uint32_t type __attribute__((ext_vector_type(2), aligned(2)));
};
template <>
struct Words<16> {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2)));
};
template <bool RAG, typename T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T *p, int n) {
    typedef typename Words<sizeof(T) * V>::type words;
    if (!RAG || n == V) {
        const words w = *reinterpret_cast<const words *>(p);
        return __builtin_bit_cast(Vec<T, V>, w);
    }
    Vec<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = i < n ? p[i] : T(0);
    return r;
}
// (NT: a nontemporal store)
template <bool RAG, bool NT = false, typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const Vec<T, V> &r, int n) {
    typedef typename Words<sizeof(T) * V>::type words;
    if (!RAG || n == V) {
        if constexpr (NT)
            __builtin_nontemporal_store(__builtin_bit_cast(words, r),
                                        reinterpret_cast<words *>(p));
        else
            *reinterpret_cast<words *>(p) = __builtin_bit_cast(words, r);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) p[i] = r.v[i];
    }
}
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return bf16_to_f32(v); }
template <typename T, int V>
__device__ __forceinline__ void widen(const Vec<T, V> &r, float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_f32(r.v[i]);
}
template <int V>
__device__ __forceinline__ Vec<float, V> narrow(const float (&f)[V], float) {
    Vec<float, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = f[i];
    return r;
}
template <int V>
__device__ __forceinline__ Vec<uint16_t, V> narrow(const float (&f)[V], uint16_t) {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    return __builtin_bit_cast(Vec<uint16_t, V>, w);
}

// The channels of vector `vec`: its output tensor, first channel there and in
// x, and how many of its V channels exist.
struct Chan {
    int seg, local, c, n;
    int width;   // channels of the output tensor
};
template <int V>
__device__ __forceinline__ Chan chan_of(int vec, const int32_t (&ch)[3]) {
    Chan r;
    r.seg = 0;
    int base = 0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int nv = (ch[s] + V - 1) / V;
        if (r.seg == s && vec >= nv) {
            vec -= nv;
            base += ch[s];
            r.seg = s + 1;
        }
    }
    r.width = r.seg == 0 ? ch[0] : (r.seg == 1 ? ch[1] : ch[2]);
    r.local = vec * V;
    r.c = base + r.local;
    r.n = min(V, r.width - r.local);
    return r;
}
template <typename P>
__device__ __forceinline__ P pick(P p0, P p1, P p2, int seg) {
    return seg == 0 ? p0 : (seg == 1 ? p1 : p2);
}

// Plain data of a launch (everything the kernels read besides the tensors).
struct ConvGeom {
    int64_t T, sxb, sxt;
    int32_t Bt, C, ch[3];
    int32_t nvec;        // lanes' vectors over the three tensors
    int32_t ntile, tt;   // runs of tokens per sequence, tokens per run
    int32_t blk;         // workgroups per sequence (fwd) or vector blocks (bwd)
    int32_t silu;
};

template <bool RAG, int W, int V>
__device__ __forceinline__ void load_weights(const float *__restrict__ weight,
                                             const float *__restrict__ bias, int c, int n,
                                             float (&w)[W][V], float (&bs)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const bool in = !RAG || i < n;
#pragma unroll
        for (int k = 0; k < W; ++k) w[k][i] = in ? weight[(int64_t)(c + i) * W + k] : 0.f;
        bs[i] = in && bias ? bias[c + i] : 0.f;
    }
}

// One run of tokens of one sequence, V channels per lane.  Tokens at or past
// the sequence's length are written as zeros.  The first run also writes the
// final state: it alone reads the initial state, so the two may be the same
// memory.
template <typename Tio, int W, bool RAG, bool NT>
__global__ __launch_bounds__(256) void conv1d_fwd_kernel(
    const Tio *__restrict__ x, const float *__restrict__ weight, const float *__restrict__ bias,
    const Tio *init, const int32_t *__restrict__ lens, Tio *__restrict__ y0,
    Tio *__restrict__ y1, Tio *__restrict__ y2, Tio *fin, ConvGeom g) {
    constexpr int V = kVec;
    const int32_t b = blockIdx.x / (uint32_t)g.blk;
    const uint32_t idx = (blockIdx.x - (uint32_t)b * g.blk) * 256u + threadIdx.x;
    if (idx >= (uint32_t)g.nvec * (uint32_t)g.ntile) return;
    const int32_t tile = idx / (uint32_t)g.nvec;
    const Chan ci = chan_of<V>(idx - (uint32_t)tile * g.nvec, g.ch);
    const Tio *xb = x + b * g.sxb + ci.c;
    const int64_t len = lens ? min((int64_t)max(lens[b], 0), g.T) : g.T;
    const int64_t t0 = (int64_t)tile * g.tt;
    const int64_t t1 = min(g.T, t0 + g.tt);
    const int64_t te = min(t1, len);

    Vec<Tio, V> head[W - 1];   // the carried state (first run only)
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        head[k] = Vec<Tio, V>{};
        if (tile == 0 && init)
            head[k] = load_vec<RAG, Tio, V>(init + ((int64_t)b * (W - 1) + k) * g.C + ci.c, ci.n);
    }

    Tio *yb = pick(y0, y1, y2, ci.seg) + (int64_t)b * g.T * ci.width + ci.local;
    if (t0 < te) {
        float w[W][V], bs[V], win[W - 1][V];
        load_weights<RAG, W, V>(weight, bias, ci.c, ci.n, w, bs);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int64_t t = t0 - (W - 1) + k;
            widen(t < 0 ? head[k] : load_vec<RAG, Tio, V>(xb + t * g.sxt, ci.n), win[k]);
        }
        // U rows in flight ahead of the arithmetic
        constexpr int U = 4;
        Vec<Tio, V> cur[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            cur[u] = load_vec<RAG, Tio, V>(xb + min(t0 + u, te - 1) * g.sxt, ci.n);
        for (int64_t t = t0; t < te; t += U) {
            Vec<Tio, V> nxt[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                nxt[u] = load_vec<RAG, Tio, V>(xb + min(t + U + u, te - 1) * g.sxt, ci.n);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t + u < te) {
                    float xv[V], out[V];
                    widen(cur[u], xv);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float p = bs[i];
#pragma unroll
                        for (int k = 0; k < W - 1; ++k) p += w[k][i] * win[k][i];
                        p += w[W - 1][i] * xv[i];
                        out[i] = g.silu ? fast_silu(p) : p;
#pragma unroll
                        for (int k = 0; k + 1 < W - 1; ++k) win[k][i] = win[k + 1][i];
                        win[W - 2][i] = xv[i];
                    }
                    store_vec<RAG, NT>(yb + (t + u) * ci.width, narrow(out, Tio(0)), ci.n);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) cur[u] = nxt[u];
        }
    }
    for (int64_t t = max(te, t0); t < t1; ++t)
        store_vec<RAG>(yb + t * ci.width, Vec<Tio, V>{}, ci.n);

    if (tile == 0 && fin) {
        Vec<Tio, V> last[W - 1];
#pragma unroll
        for (int r = 0; r < W - 1; ++r) {
            const int64_t t = len + r - (W - 1);
            if (t >= 0) {
                last[r] = load_vec<RAG, Tio, V>(xb + t * g.sxt, ci.n);
            } else {
                last[r] = Vec<Tio, V>{};
#pragma unroll
                for (int k = 0; k < W - 1; ++k)
                    if (t + (W - 1) == k) last[r] = head[k];
            }
        }
#pragma unroll
        for (int r = 0; r < W - 1; ++r)
            store_vec<RAG>(fin + ((int64_t)b * (W - 1) + r) * g.C + ci.c, last[r], ci.n);
    }
}

// One token per sequence: the window is the slot's state and the new token;
// the state moves up by one row in place.  A lane serves R sequences so that
// its weights (as many bytes as a sequence's whole traffic) are read once for
// all of them (256 sequences, 10240 channels, bf16: 8.7 us, 4.8 TB/s; float32
// 13.5 us, 6.2 TB/s, part of it from the memory-side cache).
template <typename Tio, int W, int R, bool RAG>
__global__ __launch_bounds__(256) void conv1d_step_kernel(
    Tio *__restrict__ state, const int32_t *__restrict__ slots, int64_t nslots,
    const Tio *__restrict__ x, const float *__restrict__ weight, const float *__restrict__ bias,
    Tio *__restrict__ y0, Tio *__restrict__ y1, Tio *__restrict__ y2, ConvGeom g) {
    constexpr int V = kVec;
    const uint32_t idx = blockIdx.x * 256u + threadIdx.x;
    const uint32_t grp = idx / (uint32_t)g.nvec;
    const int64_t b0 = (int64_t)grp * R;
    if (b0 >= g.Bt) return;
    const Chan ci = chan_of<V>(idx - grp * g.nvec, g.ch);
    Vec<Tio, V> row[R][W];
    int64_t base[R];
    bool live[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t b = b0 + r;
        const int64_t s = b < g.Bt ? (slots ? (int64_t)slots[b] : b) : -1;
        live[r] = s >= 0 && s < nslots;
        base[r] = s * (W - 1) * g.C + ci.c;
        if (live[r]) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                row[r][k] = load_vec<RAG, Tio, V>(state + base[r] + (int64_t)k * g.C, ci.n);
            row[r][W - 1] = load_vec<RAG, Tio, V>(x + b * g.sxb + ci.c, ci.n);
        }
    }
    float w[W][V], bs[V];
    load_weights<RAG, W, V>(weight, bias, ci.c, ci.n, w, bs);
    Tio *yp = pick(y0, y1, y2, ci.seg) + ci.local;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t b = b0 + r;
        if (b >= g.Bt) break;
        float out[V];
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = bs[i];
        if (live[r]) {
#pragma unroll
            for (int k = 0; k < W; ++k) {
                float v[V];
                widen(row[r][k], v);
#pragma unroll
                for (int i = 0; i < V; ++i) out[i] += w[k][i] * v[i];
            }
#pragma unroll
            for (int i = 0; i < V; ++i) out[i] = g.silu ? fast_silu(out[i]) : out[i];
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                store_vec<RAG>(state + base[r] + (int64_t)k * g.C, row[r][k + 1], ci.n);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) out[i] = 0.f;
        }
        store_vec<RAG>(yp + b * ci.width, narrow(out, Tio(0)), ci.n);
    }
}

// Gradients.  With dp_t = dy_t act'(pre_t):
//     dx_t = sum_j w[W-1-j] dp_{t+j},  dw[k] = sum_t dp_t x_{t-(W-1)+k},  db = sum_t dp_t.
// pre is recomputed from x.  A lane walks its run of tokens with the last W-1
// inputs and the last W-1 dp in registers, and past the run's end by W-1 more
// tokens for the dx of its last ones.  dw and db are summed in registers over
// the run, over the workgroup's 4 runs in LDS, and over the workgroups by
// conv1d_bwd_reduce_kernel, always in the same order (4 x 2048 tokens, 2304
// channels, bf16: 42 us with the 4 us of the reduction).
template <typename Tio, int W, bool RAG>
__global__ __launch_bounds__(256) void conv1d_bwd_kernel(
    const Tio *__restrict__ x, const float *__restrict__ weight, const float *__restrict__ bias,
    const Tio *__restrict__ init, const float *__restrict__ dy0, const float *__restrict__ dy1,
    const float *__restrict__ dy2, const float *__restrict__ dfinal, float *__restrict__ dx,
    float *__restrict__ dinit, float *__restrict__ part, ConvGeom g) {
    constexpr int V = kVec;
    __shared__ float red[4][(W + 1) * V][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t vb = blockIdx.x % (uint32_t)g.blk;
    const uint32_t rest = blockIdx.x / (uint32_t)g.blk;
    const uint32_t ntb = (g.ntile + 3) >> 2;
    const int32_t b = rest / ntb;
    const int32_t tile = (rest - (uint32_t)b * ntb) * 4 + wave;
    const int32_t vec = vb * 64 + lane;
    float dw[W][V] = {}, db[V] = {};
    if (vec < g.nvec && tile < g.ntile) {
        const Chan ci = chan_of<V>(vec, g.ch);
        const Tio *xb = x + b * g.sxb + ci.c;
        const float *dyb = pick(dy0, dy1, dy2, ci.seg) + (int64_t)b * g.T * ci.width + ci.local;
        const int64_t t0 = (int64_t)tile * g.tt;
        const int64_t t1 = min(g.T, t0 + g.tt);
        float w[W][V], bs[V], win[W - 1][V], dwin[W - 1][V] = {};
        load_weights<RAG, W, V>(weight, bias, ci.c, ci.n, w, bs);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int64_t t = t0 - (W - 1) + k;
            Vec<Tio, V> r = Vec<Tio, V>{};
            if (t >= 0)
                r = load_vec<RAG, Tio, V>(xb + t * g.sxt, ci.n);
            else if (init)
                r = load_vec<RAG, Tio, V>(init + ((int64_t)b * (W - 1) + k) * g.C + ci.c, ci.n);
            widen(r, win[k]);
        }
        const int64_t send = t1 + W - 1;   // dp of tokens t0 .. send-1 (0 past T)
        constexpr int U = 2;   // rows in flight ahead of the arithmetic
        struct Row {
            Vec<Tio, V> x;
            Vec<float, V> dy;
        };
        const int64_t slast = min(send, g.T);   // (rows past T are zero)
        auto load_row = [&](int64_t s) {
            Row r = Row{};
            if (s < slast) {
                r.x = load_vec<RAG, Tio, V>(xb + s * g.sxt, ci.n);
                r.dy = load_vec<RAG, float, V>(dyb + s * ci.width, ci.n);
            }
            return r;
        };
        Row cur[U];
#pragma unroll
        for (int u = 0; u < U; ++u) cur[u] = load_row(t0 + u);
        for (int64_t s0 = t0; s0 < send; s0 += U) {
            Row nxt[U];
#pragma unroll
            for (int u = 0; u < U; ++u) nxt[u] = load_row(s0 + U + u);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t s = s0 + u;
                if (s >= send) break;
                float xv[V], out[V];
                widen(cur[u].x, xv);
                const bool own = s < t1;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float dp = cur[u].dy.v[i];
                    if (g.silu) {
                        float p = bs[i];
#pragma unroll
                        for (int k = 0; k < W - 1; ++k) p += w[k][i] * win[k][i];
                        p += w[W - 1][i] * xv[i];
                        // silu' = s (1 + p (1 - s)), s = sigmoid(p); dy = 0 stays 0
                        const float sg = __builtin_amdgcn_rcpf(1.f + fast_exp2(-kLog2e * p));
                        dp *= sg * (1.f + p * (1.f - sg));
                        if (s >= g.T) dp = 0.f;
                    }
                    if (own) {
#pragma unroll
                        for (int k = 0; k < W - 1; ++k) dw[k][i] += dp * win[k][i];
                        dw[W - 1][i] += dp * xv[i];
                        db[i] += dp;
                    }
                    float d = w[0][i] * dp;
#pragma unroll
                    for (int j = 1; j < W; ++j) d += w[j][i] * dwin[W - 1 - j][i];
                    out[i] = d;
#pragma unroll
                    for (int k = 0; k + 1 < W - 1; ++k) {
                        win[k][i] = win[k + 1][i];
                        dwin[k][i] = dwin[k + 1][i];
                    }
                    win[W - 2][i] = xv[i];
                    dwin[W - 2][i] = dp;
                }
                const int64_t t = s - (W - 1);
                if (s >= g.T && dfinal) {   // token t is row s - T of the final state
                    const Vec<float, V> f = load_vec<RAG, float, V>(
                        dfinal + ((int64_t)b * (W - 1) + (s - g.T)) * g.C + ci.c, ci.n);
#pragma unroll
                    for (int i = 0; i < V; ++i) out[i] += f.v[i];
                }
                Vec<float, V> o;
#pragma unroll
                for (int i = 0; i < V; ++i) o.v[i] = out[i];
                if (t >= t0)
                    store_vec<RAG>(dx + ((int64_t)b * g.T + t) * g.C + ci.c, o, ci.n);
                else if (t < 0 && dinit)    // the first run: rows of the initial state
                    store_vec<RAG>(dinit + ((int64_t)b * (W - 1) + s) * g.C + ci.c, o, ci.n);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) cur[u] = nxt[u];
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k) red[wave][k * V + i][lane] = dw[k][i];
        red[wave][W * V + i][lane] = db[i];
    }
    __syncthreads();
    // part[rest][k][C], k = W for the bias
    float *pp = part + (int64_t)rest * (W + 1) * g.C;
    for (int e = threadIdx.x; e < (W + 1) * V * 64; e += 256) {
        const int k = e >> 8, l = (e & 255) >> 2, i = e & 3;
        const int v = vb * 64 + l;
        if (v >= g.nvec) continue;
        const Chan ci = chan_of<V>(v, g.ch);
        if (i >= ci.n) continue;
        const float *r = &red[0][k * V + i][l];
        constexpr int S = (W + 1) * V * 64;
        pp[(int64_t)k * g.C + ci.c + i] = (r[0] + r[S]) + (r[2 * S] + r[3 * S]);
    }
}

// dweight [C][W] and dbias [C] from part [np][W+1][C]: a workgroup owns 64
// channels of one tap; its 4 wavefronts take every fourth partial.
__global__ __launch_bounds__(256) void conv1d_bwd_reduce_kernel(const float *__restrict__ part,
                                                                int64_t np, int32_t C, int32_t W,
                                                                float *__restrict__ dweight,
                                                                float *__restrict__ dbias) {
    __shared__ double red[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int32_t c = blockIdx.x * 64 + lane;
    const int32_t k = blockIdx.y;
    double s = 0.0;
    if (c < C) {
        const float *p = part + (int64_t)k * C + c;
        const int64_t step = (int64_t)(W + 1) * C;
#pragma unroll 8
        for (int64_t i = wave; i < np; i += 4) s += (double)p[i * step];
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < C) {
        const float v = (float)((red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]));
        if (k < W)
            dweight[(int64_t)c * W + k] = v;
        else if (dbias)
            dbias[c] = v;
    }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

int64_t vectors(const ConvArgs &a) {
    return cdiv(a.ch[0], kVec) + cdiv(a.ch[1], kVec) + cdiv(a.ch[2], kVec);
}
// Tokens per lane: long runs reread few rows and weights, short ones fill the
// chip when there are few sequences or channels.  Forward runs of 32 where that
// leaves 2^18 lanes (half of the chip's; 8 x 4096 tokens, 5376 channels: 137 us,
// runs of 16 147, of 8 177; 4 x 2048 tokens, 2304 channels, 2^17 lanes: 20.5, runs
// of 16 19.4, of 8 21.4), runs under 16 only to reach 2^17 (1 x 1024 tokens, 5376
// channels: 9.0 us in runs of 8 and of 16, 10.6 in 4 and in 32).  Backward, where a
// lane holds twice the registers, 2^17 (4 x 2048 tokens, 2304 channels: 42 us in
// runs of 32, 46 in runs of 16).
int64_t run_length(const ConvArgs &a, int64_t lanes) {
    int64_t tt = 32;
    while (tt > 4 &&
           a.Bt * vectors(a) * cdiv(a.T, tt) < (tt > 16 ? lanes : int64_t(1) << 17))
        tt >>= 1;
    return tt;
}
int64_t fwd_run(const ConvArgs &a) { return run_length(a, int64_t(1) << 18); }
int64_t bwd_run(const ConvArgs &a) { return run_length(a, int64_t(1) << 17); }

ConvGeom geom(const ConvArgs &a, int64_t tt) {
    ConvGeom g;
    g.T = a.T;
    g.sxb = a.sxb;
    g.sxt = a.sxt;
    g.Bt = (int32_t)a.Bt;
    g.C = (int32_t)a.C;
    for (int i = 0; i < 3; ++i) g.ch[i] = (int32_t)a.ch[i];
    g.nvec = (int32_t)vectors(a);
    g.tt = (int32_t)tt;
    g.ntile = (int32_t)(a.T > 0 ? cdiv(a.T, tt) : 1);
    g.blk = 0;
    g.silu = a.silu ? 1 : 0;
    return g;
}

// f(integral_constant<W>, bool_constant<RAG>) for the launch's taps, and
// whether some tensor's channels end inside a lane's vector.
template <typename F>
void by_width(const ConvArgs &a, F f) {
    const bool rag = a.ch[0] % kVec || a.ch[1] % kVec || a.ch[2] % kVec;
    auto g = [&](auto w) {
        if (rag)
            f(w, std::true_type());
        else
            f(w, std::false_type());
    };
    if (a.W == 2) g(std::integral_constant<int, 2>());
    if (a.W == 3) g(std::integral_constant<int, 3>());
    if (a.W == 4) g(std::integral_constant<int, 4>());
}

// Outputs that outgrow the 256 MB memory-side cache are not found there by the
// scan that reads them next: nontemporal stores (8 x 4096 tokens, 5376 channels,
// 352 MB: 137 us, plain 149).  Smaller ones stay cached.
bool streams(const ConvArgs &a) {
    return a.Bt * a.T * a.C * (a.bf16 ? 2 : 4) > (int64_t(256) << 20);
}

template <typename Tio>
void fwd_t(const ConvArgs &a, const ConvGeom &g, hipStream_t st) {
    by_width(a, [&](auto w, auto rag) {
        auto launch = [&](auto nt) {
            conv1d_fwd_kernel<Tio, decltype(w)::value, decltype(rag)::value, decltype(nt)::value>
                <<<dim3((uint32_t)(a.Bt * g.blk)), 256, 0, st>>>(
                    (const Tio *)a.x, a.weight, a.bias, (const Tio *)a.init, a.lens,
                    (Tio *)a.y[0], (Tio *)a.y[1], (Tio *)a.y[2], (Tio *)a.fin, g);
        };
        if (streams(a))
            launch(std::true_type());
        else
            launch(std::false_type());
    });
}

template <typename Tio, int R>
void step_r(const ConvArgs &a, const ConvGeom &g, hipStream_t st) {
    const dim3 grid((uint32_t)cdiv(cdiv(a.Bt, R) * g.nvec, 256));
    by_width(a, [&](auto w, auto rag) {
        conv1d_step_kernel<Tio, decltype(w)::value, R, decltype(rag)::value>
            <<<grid, 256, 0, st>>>((Tio *)a.state, a.slots, a.nslots, (const Tio *)a.x, a.weight,
                                   a.bias, (Tio *)a.y[0], (Tio *)a.y[1], (Tio *)a.y[2], g);
    });
}
// 4 sequences per lane where that still leaves a wavefront on every other
// SIMD (10240 channels: 256 sequences 8.7 us, one per lane 11.2; 64: 4.7 both; but
// 32, a wavefront on a third of them: 4.3, 3.8)
int step_rows(const ConvArgs &a) { return a.Bt * vectors(a) >= int64_t(1) << 17 ? 4 : 1; }
template <typename Tio>
void step_t(const ConvArgs &a, const ConvGeom &g, hipStream_t st) {
    if (step_rows(a) == 4)
        step_r<Tio, 4>(a, g, st);
    else
        step_r<Tio, 1>(a, g, st);
}

template <typename Tio>
void bwd_t(const ConvArgs &a, const ConvGeom &g, int64_t parts, hipStream_t st) {
    by_width(a, [&](auto w, auto rag) {
        conv1d_bwd_kernel<Tio, decltype(w)::value, decltype(rag)::value>
            <<<dim3((uint32_t)(parts * g.blk)), 256, 0, st>>>(
                (const Tio *)a.x, a.weight, a.bias, (const Tio *)a.init, a.dy[0], a.dy[1], a.dy[2],
                a.dfinal, a.dx, a.dinit, a.part, g);
    });
}

int64_t bwd_parts(const ConvArgs &a) {
    return a.Bt * cdiv(a.T > 0 ? cdiv(a.T, bwd_run(a)) : 1, 4);
}

}  // namespace

bool conv1d_fits(const ConvArgs &a) {
    const double nvec = (double)vectors(a), T = a.T > 0 ? (double)a.T : 1.0, Bt = (double)a.Bt;
    const double fwd = Bt * (nvec * (T / (double)fwd_run(a) + 1.0) / 256.0 + 1.0);
    const double bwd = Bt * (T / (4.0 * (double)bwd_run(a)) + 1.0) * (nvec / 64.0 + 1.0);
    const double step = Bt * nvec / 256.0 + 1.0;
    const double most = (double)kMaxBlocks;
    return fwd <= most && bwd <= most && step <= most;
}

ConvLayout conv1d_layout(const ConvArgs &a) {
    return ConvLayout{fwd_run(a), bwd_run(a), step_rows(a)};
}

hipError_t launch_conv1d_fwd(const ConvArgs &a, hipStream_t st) {
    ConvGeom g = geom(a, fwd_run(a));
    g.blk = (int32_t)cdiv((int64_t)g.nvec * g.ntile, 256);
    if (a.bf16)
        fwd_t<uint16_t>(a, g, st);
    else
        fwd_t<float>(a, g, st);
    return hipGetLastError();
}

hipError_t launch_conv1d_step(const ConvArgs &a, hipStream_t st) {
    const ConvGeom g = geom(a, 1);
    if (a.bf16)
        step_t<uint16_t>(a, g, st);
    else
        step_t<float>(a, g, st);
    return hipGetLastError();
}

size_t conv1d_bwd_workspace(const ConvArgs &a) {
    return (size_t)bwd_parts(a) * (a.W + 1) * a.C * sizeof(float);
}

hipError_t launch_conv1d_bwd(const ConvArgs &a, hipStream_t st) {
    ConvGeom g = geom(a, bwd_run(a));
    g.blk = (int32_t)cdiv(g.nvec, 64);
    const int64_t parts = bwd_parts(a);
    if (parts > 0) {   // (no sequences: the sums below are zero)
        if (a.bf16)
            bwd_t<uint16_t>(a, g, parts, st);
        else
            bwd_t<float>(a, g, parts, st);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    conv1d_bwd_reduce_kernel<<<dim3((uint32_t)cdiv(a.C, 64), (uint32_t)(a.W + 1)), 256, 0, st>>>(
        a.part, parts, (int32_t)a.C, (int32_t)a.W, a.dweight, a.dbias);
    return hipGetLastError();
}

}  // namespace ssd
