// C ABI of the gradients (include/ssm.h): argument checks, the workspace's layout and the
// launches of a backward pass. Nothing here allocates, frees or synchronises.
#include <algorithm>

#include "api_common.h"
#include "bwd_launch.h"

namespace {

using namespace ssm;

constexpr int kNumSMs = 148;

struct BwdPlan {
    int lanes;
    BwdVariant v;
    int groups, nseg, seg_len, nsub, conv_chunks;
    // byte offsets of the workspace's parts
    size_t ckpt, parts, pA, pA_lo, pD, sumP, sumS, sumR, since, du32, conv_part, total;
};

// Time of `ctas` CTAs on the GPU, in that of one alone on an SM. Up to per_sm share one, and k of
// them take 1 + share (k - 1) times as long as one alone: they wait for one another's latencies
// rather than for a pipe.
double waves(int64_t ctas, int per_sm, double share) {
    const int64_t full = ctas / (kNumSMs * per_sm), rest = ctas % (kNumSMs * per_sm);
    const int64_t k = (rest + kNumSMs - 1) / kNumSMs;
    return full * (1 + share * (per_sm - 1)) + (rest ? 1 + share * (k - 1) : 0);
}

// Time (us) of a backward pass in n segments of per tiles, one more to fill and drain each: 0.65
// of a tile's time is the sweep's, 0.35 the checkpoint pass's, which runs with twice the CTAs an
// SM; segments add the summary pass, as long, and the chain. A tile's time in us, by lanes a
// channel (d_state 1..4, 8, 16 (tiles of 16 steps), 32, 64, 128), of one CTA an SM.
double sweep_time(const BwdVariant& v, int lanes, int64_t ctas, int64_t per, int64_t n) {
    const double tile = lanes == 1 ? 3.3 : lanes == 2 ? 2.5 : lanes == 4 ? 4.4 : lanes == 8 ? 2.7 : lanes == 16 ? 7.5 : 16;
    return tile * (per + 1) *
               (0.65 * waves(ctas * n, v.ctas, 0.7) + 0.35 * (n > 1 ? 2 : 1) * waves(ctas * n, 2 * v.ctas, 0.35)) +
           (n > 1 ? 0.6 * n : 0);
}

ssm_status_t plan_bwd(const ssm_scan_bwd_args_t* a, BwdPlan* pl) {
    if (!a) return api_fail(SSM_ERR_NULL_ARG, "args is NULL");
    if (bad_dtype(a->dtype))
        return api_fail(SSM_ERR_BAD_DTYPE, "dtype %d is not SSM_F32 or SSM_BF16", (int)a->dtype);
    if (a->batch < 0 || a->dim < 0 || a->seqlen < 0) return api_fail(SSM_ERR_BAD_SHAPE, "negative size");
    if (a->dstate < 1 || a->dstate > SSM_MAX_SCAN_DSTATE)
        return api_fail(SSM_ERR_BAD_SHAPE, "dstate %lld outside 1..%d", (long long)a->dstate,
                        SSM_MAX_SCAN_DSTATE);
    if (a->a_heads < 0 || (a->a_heads > 0 && a->dim % a->a_heads != 0))
        return api_fail(SSM_ERR_BAD_SHAPE, "a_heads %d must be 0 or divide dim %lld", a->a_heads,
                        (long long)a->dim);
    if (a->seqlen > 0x3fffffffLL || a->dim > 0x3fffffffLL)
        return api_fail(SSM_ERR_BAD_SHAPE, "seqlen and dim must be below 2^30");
    if (a->batch > 65535) return api_fail(SSM_ERR_UNSUPPORTED, "batch %lld > 65535", (long long)a->batch);
    if (a->batch * a->dim > 0x7fffffffLL)
        return api_fail(SSM_ERR_BAD_SHAPE, "batch * dim must be below 2^31");
    if ((double)a->batch * (double)a->dim * (double)a->seqlen > 1099511627776.0)
        return api_fail(SSM_ERR_BAD_SHAPE, "batch * dim * seqlen exceeds 2^40");
    if (a->conv_weight && (a->conv_width < 1 || a->conv_width > SSM_MAX_CONV_WIDTH))
        return api_fail(SSM_ERR_BAD_SHAPE, "conv_width %d outside 1..%d", a->conv_width,
                        SSM_MAX_CONV_WIDTH);
    if (a->num_segments < 0) return api_fail(SSM_ERR_BAD_SHAPE, "num_segments %d < 0", a->num_segments);
    if (a->reverse && (a->initial_state || a->conv_history || a->dinitial_state))
        return api_fail(SSM_ERR_UNSUPPORTED,
                        "initial_state, conv_history and dinitial_state need a forward scan");
    if (!a->conv_weight && (a->conv_history || a->dconv_weight || a->dconv_bias))
        return api_fail(SSM_ERR_NULL_ARG, "conv_history, dconv_weight and dconv_bias need conv_weight");
    if (a->dconv_history && !a->conv_history)
        return api_fail(SSM_ERR_NULL_ARG, "dconv_history needs conv_history");
    if (a->dz && !a->z) return api_fail(SSM_ERR_NULL_ARG, "dz needs z");
    if ((a->u_scale != nullptr) != (a->delta_scale != nullptr) ||
        (a->u_scale != nullptr && a->z) != (a->z_scale != nullptr))
        return api_fail(SSM_ERR_NULL_ARG, "u, delta and z are all packed or none: scales missing");
    if (a->channel_last) {
        struct { int64_t s, w; const char* n; } sd[] = {
            {a->stride_u, a->dim, "stride_u"}, {a->stride_delta, a->dim, "stride_delta"},
            {a->stride_z, a->dim, "stride_z"}, {a->stride_dout, a->dim, "stride_dout"},
            {a->stride_B, a->dstate, "stride_B"}, {a->stride_C, a->dstate, "stride_C"},
            {a->stride_du, a->dim, "stride_du"}, {a->stride_ddelta, a->dim, "stride_ddelta"},
            {a->stride_dz, a->dim, "stride_dz"}, {a->stride_dB, a->dstate, "stride_dB"},
            {a->stride_dC, a->dstate, "stride_dC"}};
        for (auto& x : sd)
            if (x.s != 0 && (x.s < x.w || x.s > (1ll << 31)))
                return api_fail(SSM_ERR_BAD_SHAPE, "%s %lld: 0 or from %lld to 2^31", x.n,
                                (long long)x.s, (long long)x.w);
    }
    if (a->seq_starts) {
        if (a->num_seqs < 1 || a->num_seqs > 0x3fffffff)
            return api_fail(SSM_ERR_BAD_SHAPE, "num_seqs %d < 1", a->num_seqs);
        if (a->batch != 1)
            return api_fail(SSM_ERR_UNSUPPORTED, "packed sequences need batch 1 (got %lld)",
                            (long long)a->batch);
        if (a->reverse || a->initial_state || a->conv_history || a->dfinal_state ||
            a->dinitial_state || a->a_heads > 0)
            return api_fail(SSM_ERR_UNSUPPORTED,
                            "packed sequences: forward scans with per-state A, without states or history");
    }

    const int64_t Bn = a->batch, D = a->dim, L = a->seqlen;
    pl->lanes = 1;
    while (4 * pl->lanes < a->dstate) pl->lanes *= 2;
    pl->v = scan_bwd_variant(pl->lanes, size_of(a->dtype), a->a_heads > 0);
    const int64_t tile = pl->v.tile, ntiles = std::max<int64_t>(1, (L + tile - 1) / tile);
    pl->groups = (int)((D + pl->v.channels - 1) / pl->v.channels);
    // Segments: the number that the model above finds fastest. Segments fill SMs that one CTA per
    // row and channel group leaves idle, or even out the last wave; they cost a second forward pass
    // and the chain over them. Measured against 1 to 40 segments, 14 kernels at 8 shapes of over
    // 80 us, the choice is 0.9 % off the best on average, at most 7 % (bf16 B8 D1536 L2048 N16:
    // one sweep 0.89 ms, 1.07 in 3 segments; fp32 B4 D1536 L2048 N128: 6.98 in one, 5.97 in 3;
    // bf16 B1 D3840 L8192 N16: 2.20 in one, 1.27 in 16).
    int64_t nseg = a->num_segments;
    if (nseg == 0) {
        const int64_t ctas = pl->groups * Bn, slots = (int64_t)kNumSMs * pl->v.ctas;
        nseg = 1;
        if (ctas > 0) {
            double best = 1e30;
            const int64_t most = std::max<int64_t>(1, std::min<int64_t>(8 * slots / ctas, 1024));
            for (int64_t per = ntiles;; --per) {               // once for each number that differs
                const int64_t n = (ntiles + per - 1) / per;
                if (n > most) break;
                per = (ntiles + n - 1) / n;
                const double t = sweep_time(pl->v, pl->lanes, ctas, per, n);
                if (t < best) {
                    best = t;
                    nseg = n;
                }
                if (per == 1) break;
            }
        }
    }
    nseg = std::max<int64_t>(1, std::min<int64_t>({nseg, ntiles, 4096}));
    const int64_t per = (ntiles + nseg - 1) / nseg;
    pl->seg_len = (int)std::min<int64_t>(per * tile, 0x40000000);
    pl->nseg = (int)((ntiles + per - 1) / per);
    pl->nsub = (int)(ntiles * tile / pl->v.steps);
    const int chunk = conv_bwd_chunk(a->channel_last != 0);
    pl->conv_chunks = (int)((L + chunk - 1) / chunk);

    size_t at = 0;
    auto take = [&](size_t n, size_t* off) {
        *off = at;
        at += (n + 255) / 256 * 256;
    };
    const size_t ns = pl->v.ns, rows = (size_t)pl->nseg * Bn;
    const bool empty = Bn * D * L == 0;
    const size_t dns = (size_t)D * ns * 4;
    take(empty ? 0 : (size_t)Bn * pl->nsub * dns, &pl->ckpt);
    take(empty ? 0 : (size_t)pl->groups * Bn * L * 2 * ns * 4, &pl->parts);
    take(empty ? 0 : rows * dns, &pl->pA);
    take(empty || per <= pl->v.drain ? 0 : rows * dns, &pl->pA_lo);
    take(empty ? 0 : rows * D * 8, &pl->pD);
    const size_t sum = empty || pl->nseg == 1 ? 0 : rows * dns;
    take(sum, &pl->sumP);
    take(sum, &pl->sumS);
    take(sum, &pl->sumR);
    take(empty || !a->seq_starts ? 0 : (size_t)L, &pl->since);
    take(empty || !a->conv_weight ? 0 : (size_t)Bn * D * L * 4, &pl->du32);
    take(empty || !a->conv_weight ? 0 : (size_t)Bn * pl->conv_chunks * D * 20, &pl->conv_part);
    pl->total = at;
    return SSM_OK;
}

}  // namespace

extern "C" {

ssm_status_t ssm_selective_scan_bwd_workspace_size(const ssm_scan_bwd_args_t* a, size_t* bytes) {
    if (!bytes) return api_fail(SSM_ERR_NULL_ARG, "bytes is NULL");
    BwdPlan pl;
    ssm_status_t st = plan_bwd(a, &pl);
    if (st != SSM_OK) return st;
    *bytes = pl.total;
    return api_ok();
}

ssm_status_t ssm_selective_scan_bwd(const ssm_scan_bwd_args_t* a, ssm_stream_t stream) {
    BwdPlan pl;
    ssm_status_t status = plan_bwd(a, &pl);
    if (status != SSM_OK) return status;
    const int64_t Bn = a->batch, D = a->dim, L = a->seqlen, N = a->dstate;
    const bool cl = a->channel_last != 0, empty = Bn * D * L == 0, packed8 = a->u_scale != nullptr;
    const size_t es = size_of(a->dtype), ein = packed8 ? 1 : es;
    const int64_t nb = (L + kBlock8 - 1) / kBlock8;

    // element strides: (batch, width, seqlen) dense, or channel-last with position stride st
    auto str = [&](int64_t st, int64_t width) {
        const int64_t s = st ? st : width;
        return cl ? Str{L * s, 1, s} : Str{width * L, L, 1};
    };
    auto span = [&](int64_t st, int64_t width, size_t size) -> size_t {
        if (Bn * L * width == 0) return 0;
        return cl ? (size_t)((Bn * L - 1) * (st ? st : width) + width) * size : (size_t)(Bn * width * L) * size;
    };
    const size_t st_bytes = (size_t)Bn * D * N * 4, sc_bytes = (size_t)Bn * D * nb * 4;
    const size_t hist_bytes = a->conv_weight ? (size_t)Bn * D * (a->conv_width - 1) * es : 0;
    const size_t a_bytes = (a->a_heads > 0 ? (size_t)a->a_heads : (size_t)D * N) * 4;
    const size_t w_bytes = a->conv_weight ? (size_t)D * a->conv_width * 4 : 0;
    // a view in rows, dense ones without a step
    auto view = [&](const void* q, int64_t st, int64_t width, size_t size, const char* name) {
        return cl ? Arg{q, size, span(st, width, size), name, (size_t)width * size, (size_t)(st ? st : width) * size}
                  : Arg{q, size, span(st, width, size), name};
    };
    const Arg ins[] = {
        view(a->u, a->stride_u, D, ein, "u"), view(a->delta, a->stride_delta, D, ein, "delta"),
        view(a->z, a->stride_z, D, ein, "z"), view(a->B, a->stride_B, N, es, "B"),
        view(a->C, a->stride_C, N, es, "C"), view(a->dout, a->stride_dout, D, es, "dout"),
        {a->A, 4, a_bytes, "A"},
        {a->D, 4, (size_t)D * 4, "D"}, {a->delta_bias, 4, (size_t)D * 4, "delta_bias"},
        {a->conv_weight, 4, w_bytes, "conv_weight"}, {a->conv_bias, 4, (size_t)D * 4, "conv_bias"},
        {a->initial_state, 4, st_bytes, "initial_state"}, {a->dfinal_state, 4, st_bytes, "dfinal_state"},
        {a->conv_history, es, hist_bytes, "conv_history"},
        {a->seq_starts, 4, a->seq_starts ? ((size_t)a->num_seqs + 1) * 4 : 0, "seq_starts"},
        {a->u_scale, 4, sc_bytes, "u_scale"}, {a->delta_scale, 4, sc_bytes, "delta_scale"},
        {a->z_scale, 4, sc_bytes, "z_scale"}};
    const Arg outs[] = {
        view(a->du, a->stride_du, D, es, "du"), view(a->ddelta, a->stride_ddelta, D, es, "ddelta"),
        view(a->dz, a->stride_dz, D, es, "dz"), view(a->dB, a->stride_dB, N, es, "dB"),
        view(a->dC, a->stride_dC, N, es, "dC"),
        {a->dA, 4, a_bytes, "dA"}, {a->dD, 4, (size_t)D * 4, "dD"},
        {a->ddelta_bias, 4, (size_t)D * 4, "ddelta_bias"},
        {a->dconv_weight, 4, w_bytes, "dconv_weight"}, {a->dconv_bias, 4, (size_t)D * 4, "dconv_bias"},
        {a->dinitial_state, 4, st_bytes, "dinitial_state"},
        {a->dconv_history, es, hist_bytes, "dconv_history"}, {a->workspace, 16, pl.total, "workspace"}};
    if (!empty) {
        struct { const void* p; const char* n; } req[] = {
            {a->u, "u"}, {a->delta, "delta"}, {a->A, "A"}, {a->B, "B"}, {a->C, "C"}, {a->dout, "dout"},
            {a->du, "du"}, {a->ddelta, "ddelta"}, {a->dA, "dA"}, {a->dB, "dB"}, {a->dC, "dC"}};
        for (auto& r : req)
            if (!r.p) return api_fail(SSM_ERR_NULL_ARG, "%s is NULL", r.n);
    }
    if ((status = check_aligned(ins)) != SSM_OK) return status;
    if ((status = check_aligned(outs)) != SSM_OK) return status;
    if (pl.total > 0 && (!a->workspace || a->workspace_bytes < pl.total))
        return api_fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", pl.total,
                        a->workspace ? a->workspace_bytes : (size_t)0);
    if ((status = check_alias(outs, ins)) != SSM_OK) return status;
    if ((status = check_distinct(outs)) != SSM_OK) return status;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (empty) {
        // no steps: sums over nothing, and the last state is the initial state
        auto zero = [&](void* p, size_t n) {
            if (p && n && e == cudaSuccess) e = cudaMemsetAsync(p, 0, n, s);
        };
        zero(a->dA, a_bytes);
        zero(a->dD, (size_t)D * 4);
        zero(a->ddelta_bias, (size_t)D * 4);
        zero(a->dconv_weight, w_bytes);
        zero(a->dconv_bias, (size_t)D * 4);
        zero(a->dconv_history, hist_bytes);
        struct { void* p; int64_t st; } bc[] = {{a->dB, a->stride_dB}, {a->dC, a->stride_dC}};
        for (auto& x : bc)
            if (x.p && Bn * L > 0 && e == cudaSuccess) {
                if (cl) e = cudaMemset2DAsync(x.p, (x.st ? x.st : N) * es, 0, N * es, Bn * L, s);
                else e = cudaMemsetAsync(x.p, 0, (size_t)Bn * N * L * es, s);
            }
        if (a->dinitial_state && st_bytes && e == cudaSuccess) {
            e = a->dfinal_state ? cudaMemcpyAsync(a->dinitial_state, a->dfinal_state, st_bytes,
                                                  cudaMemcpyDeviceToDevice, s)
                                : cudaMemsetAsync(a->dinitial_state, 0, st_bytes, s);
        }
        return e == cudaSuccess ? api_ok() : api_cuda(e, "zero-size gradients");
    }

    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    auto f = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
    const Str sscale = cl ? Str{nb * D, 1, D} : Str{D * nb, nb, 1};
    BwdParams p{};
    p.batch = (int)Bn;
    p.dim = (int)D;
    p.seqlen = (int)L;
    p.dstate = (int)N;
    p.x = {a->u, a->u_scale, str(a->stride_u, D), sscale};
    p.dt = {a->delta, a->delta_scale, str(a->stride_delta, D), sscale};
    p.z = {a->z, a->z_scale, str(a->stride_z, D), sscale};
    p.dy = a->dout;
    p.Bm = a->B;
    p.Cm = a->C;
    p.sdy = str(a->stride_dout, D);
    p.sB = str(a->stride_B, N);
    p.sC = str(a->stride_C, N);
    p.A = a->A;
    p.D = a->D;
    p.dbias = a->delta_bias;
    p.conv_w = a->conv_weight;
    p.conv_b = a->conv_weight ? a->conv_bias : nullptr;
    p.conv_width = a->conv_weight ? a->conv_width : 0;
    p.softplus = a->delta_softplus ? 1 : 0;
    p.reverse = a->reverse ? 1 : 0;
    p.head_dim = a->a_heads > 0 ? (int)(D / a->a_heads) : 0;
    // Asynchronous copies take 16 bytes (8 of 8-bit rows in 8-step tiles) of a row at a time,
    // from tile boundaries counted from either end of the row: bases aligned to 16 bytes, rows
    // of a multiple of 16 bytes (8-bit rows along the positions: of 16 codes, which every
    // boundary is a multiple of too).
    const int64_t unit = 16 / es, unit_in = 16 / ein;
    bool async = is_aligned(a->u, 16) && is_aligned(a->delta, 16) && is_aligned(a->z, 16) &&
                 is_aligned(a->B, 16) && is_aligned(a->C, 16) && is_aligned(a->dout, 16);
    if (cl)
        async = async && p.x.s.p % unit_in == 0 && p.dt.s.p % unit_in == 0 &&
                (!a->z || p.z.s.p % unit_in == 0) && p.sdy.p % unit == 0 && p.sB.p % unit == 0 &&
                p.sC.p % unit == 0;
    else
        async = async && L % unit == 0 && L % unit_in == 0;
    p.async = async ? 1 : 0;
    p.h0 = a->initial_state;
    p.dhl = a->dfinal_state;
    p.hist = a->conv_weight ? a->conv_history : nullptr;
    p.since = a->seq_starts ? ws + pl.since : nullptr;
    p.du = a->du;
    p.du32 = a->conv_weight ? f(pl.du32) : nullptr;
    p.sdu = a->conv_weight ? str(0, D) : str(a->stride_du, D);
    p.ddt = a->ddelta;
    p.dz = a->dz;
    p.sddt = str(a->stride_ddelta, D);
    p.sdz = str(a->stride_dz, D);
    // A thread's outputs are runs of up to 16 bytes (fp32: 32), from multiples of their length.
    bool vec = is_aligned(a->du, 16) && is_aligned(a->ddelta, 16) && is_aligned(a->dz, 16);
    if (cl) vec = vec && p.sdu.p % 8 == 0 && p.sddt.p % 8 == 0 && (!a->dz || p.sdz.p % 8 == 0);
    else vec = vec && L % 8 == 0;
    p.vec_out = vec ? 1 : 0;
    p.dh0 = a->dinitial_state;
    p.ckpt = f(pl.ckpt);
    p.nsub = pl.nsub;
    p.parts = f(pl.parts);
    p.pA = f(pl.pA);
    p.pA_lo = f(pl.pA_lo);
    p.pD = f(pl.pD);
    p.sumP = f(pl.sumP);
    p.sumS = f(pl.sumS);
    p.sumR = f(pl.sumR);
    p.nseg = pl.nseg;
    p.seg_len = pl.seg_len;

    const bool heads = a->a_heads > 0;
    using Launch = cudaError_t (*)(int, int, bool, const BwdParams&, cudaStream_t);
    static constexpr Launch kLaunch[2][2][2] = {               // bf16?, channel-last?, 8 bits?
        {{launch_scan_bwd_f32, launch_scan_bwd_f32_q8}, {launch_scan_bwd_f32_cl, launch_scan_bwd_f32_cl_q8}},
        {{launch_scan_bwd_bf16, launch_scan_bwd_bf16_q8}, {launch_scan_bwd_bf16_cl, launch_scan_bwd_bf16_cl_q8}}};
    auto scan = [&](int what) { return kLaunch[es == 2][cl][packed8](what, pl.lanes, heads, p, s); };
    if (a->seq_starts &&
        (e = launch_since(a->seq_starts, a->num_seqs, (int)L, ws + pl.since, s)) != cudaSuccess)
        return api_cuda(e, "sequence starts launch");
    if (pl.nseg > 1) {
        if ((e = scan(1)) != cudaSuccess) return api_cuda(e, "segment summary launch");
        if ((e = launch_scan_bwd_carry(pl.v.ns, p, s)) != cudaSuccess)
            return api_cuda(e, "segment carry launch");
    }
    if ((e = scan(0)) != cudaSuccess) return api_cuda(e, "state checkpoint launch");
    if ((e = scan(2)) != cudaSuccess) return api_cuda(e, "backward sweep launch");

    BwdReduceParams r{};
    r.batch = (int)Bn;
    r.dim = (int)D;
    r.seqlen = (int)L;
    r.dstate = (int)N;
    r.ns = pl.v.ns;
    r.groups = pl.groups;
    r.nrows = (int)(pl.nseg * Bn);
    r.reverse = p.reverse;
    r.head_dim = p.head_dim;
    r.order_shift = pl.v.order_shift;
    r.order_mask = pl.v.order_mask;
    r.parts = p.parts;
    r.pA = p.pA;
    r.pD = p.pD;
    r.dB = a->dB;
    r.dC = a->dC;
    r.sdB = str(a->stride_dB, N);
    r.sdC = str(a->stride_dC, N);
    r.dA = a->dA;
    r.dD = a->dD;
    r.dbias = a->ddelta_bias;
    if ((e = launch_scan_bwd_reduce((int)es, r, s)) != cudaSuccess)
        return api_cuda(e, "gradient reduction launch");

    if (a->conv_weight) {
        ConvBwdParams c{};
        c.batch = (int)Bn;
        c.dim = (int)D;
        c.seqlen = (int)L;
        c.width = a->conv_width;
        c.x = p.x;
        c.dout = p.du32;
        c.dout32 = 1;
        c.sdo = p.sdu;
        c.w = a->conv_weight;
        c.bias = p.conv_b;
        c.silu = 1;
        c.reverse = p.reverse;
        c.hist = p.hist;
        c.since = p.since;
        c.dx = a->du;
        c.sdx = str(a->stride_du, D);
        c.dhist = a->dconv_history;
        c.part = f(pl.conv_part);
        c.chunks = pl.conv_chunks;
        c.chunk_len = conv_bwd_chunk(cl);
        // runs of 16 positions (8-bit: from multiples of 16, so each within one block), or
        // channel-last of 4 channels
        c.vec = is_aligned(a->u, 16) && is_aligned(a->du, 16) &&
                (cl ? (p.x.s.p % 4 == 0 && c.sdx.p % 4 == 0 && D % 4 == 0) : (L % (packed8 ? 16 : 8) == 0));
        if ((e = launch_conv_bwd((int)es, cl, c, s)) != cudaSuccess)
            return api_cuda(e, "conv gradient launch");
        ConvReduceParams cr{(int)D, a->conv_width, Bn * pl.conv_chunks, c.part,
                            a->dconv_weight, a->dconv_bias};
        if ((a->dconv_weight || a->dconv_bias) && (e = launch_conv_reduce(cr, s)) != cudaSuccess)
            return api_cuda(e, "conv reduction launch");
    }
    return api_ok();
}

ssm_status_t ssm_causal_conv1d_bwd_workspace_size(int64_t batch, int64_t dim, int64_t seqlen,
                                                  size_t* bytes) {
    if (!bytes) return api_fail(SSM_ERR_NULL_ARG, "bytes is NULL");
    if (batch < 0 || dim < 0 || seqlen < 0) return api_fail(SSM_ERR_BAD_SHAPE, "negative size");
    if (seqlen > 0x3fffffffLL || dim > 0x3fffffffLL || batch > 0x3fffffffLL)
        return api_fail(SSM_ERR_BAD_SHAPE, "batch, seqlen and dim must be below 2^30");
    if (batch * dim > 0x7fffffffLL)
        return api_fail(SSM_ERR_BAD_SHAPE, "batch * dim must be below 2^31");
    if ((double)batch * (double)dim * (double)seqlen > 1099511627776.0)
        return api_fail(SSM_ERR_BAD_SHAPE, "batch * dim * seqlen exceeds 2^40");
    const int chunk = conv_bwd_chunk(false);
    *bytes = (size_t)batch * ((seqlen + chunk - 1) / chunk) * dim * 20;
    return api_ok();
}

ssm_status_t ssm_causal_conv1d_bwd(const void* dout, const void* x, const float* w, const float* bias,
                                   void* dx, float* dw, float* dbias, int64_t batch, int64_t dim,
                                   int64_t seqlen, int32_t width, int32_t apply_silu,
                                   ssm_dtype_t dtype, void* workspace, size_t workspace_bytes,
                                   ssm_stream_t stream) {
    if (bad_dtype(dtype))
        return api_fail(SSM_ERR_BAD_DTYPE, "dtype %d is not SSM_F32 or SSM_BF16", (int)dtype);
    size_t need = 0;
    ssm_status_t status = ssm_causal_conv1d_bwd_workspace_size(batch, dim, seqlen, &need);
    if (status != SSM_OK) return status;
    if (width < 1 || width > SSM_MAX_CONV_WIDTH)
        return api_fail(SSM_ERR_BAD_SHAPE, "width %d outside 1..%d", width, SSM_MAX_CONV_WIDTH);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t es = size_of(dtype), n = (size_t)batch * dim * seqlen * es;
    if (n == 0) {
        cudaError_t e = cudaSuccess;
        if (dw && dim) e = cudaMemsetAsync(dw, 0, (size_t)dim * width * 4, s);
        if (dbias && dim && e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, (size_t)dim * 4, s);
        return e == cudaSuccess ? api_ok() : api_cuda(e, "zero-size gradients");
    }
    if (!dout || !x || !w || !dx)
        return api_fail(SSM_ERR_NULL_ARG, "%s is NULL", !dout ? "dout" : !x ? "x" : !w ? "w" : "dx");
    const Arg ins[] = {{dout, es, n, "dout"}, {x, es, n, "x"}, {w, 4, (size_t)dim * width * 4, "w"},
                       {bias, 4, (size_t)dim * 4, "bias"}};
    const Arg outs[] = {{dx, es, n, "dx"}, {dw, 4, (size_t)dim * width * 4, "dw"},
                        {dbias, 4, (size_t)dim * 4, "dbias"}, {workspace, 16, need, "workspace"}};
    if ((status = check_aligned(ins)) != SSM_OK) return status;
    if ((status = check_aligned(outs)) != SSM_OK) return status;
    if (!workspace || workspace_bytes < need)
        return api_fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                        workspace ? workspace_bytes : (size_t)0);
    if ((status = check_alias(outs, ins)) != SSM_OK) return status;
    if ((status = check_distinct(outs)) != SSM_OK) return status;
    const Str str{dim * seqlen, seqlen, 1};
    ConvBwdParams c{};
    c.batch = (int)batch;
    c.dim = (int)dim;
    c.seqlen = (int)seqlen;
    c.width = width;
    c.x = {x, nullptr, str, {}};
    c.dout = dout;
    c.sdo = str;
    c.w = w;
    c.bias = bias;
    c.silu = apply_silu ? 1 : 0;
    c.dx = dx;
    c.sdx = str;
    c.part = static_cast<float*>(workspace);
    c.chunk_len = conv_bwd_chunk(false);
    c.chunks = (int)((seqlen + c.chunk_len - 1) / c.chunk_len);
    c.vec = seqlen % 8 == 0 && is_aligned(x, 16) && is_aligned(dout, 16) && is_aligned(dx, 16);
    cudaError_t e = launch_conv_bwd((int)es, false, c, s);
    if (e != cudaSuccess) return api_cuda(e, "conv gradient launch");
    if (dw || dbias) {
        ConvReduceParams cr{(int)dim, width, batch * c.chunks, c.part, dw, dbias};
        if ((e = launch_conv_reduce(cr, s)) != cudaSuccess) return api_cuda(e, "conv reduction launch");
    }
    return api_ok();
}

}  // extern "C"
