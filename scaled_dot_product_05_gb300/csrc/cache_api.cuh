// cache_api.cuh -- C ABI of the norm / rotation, cache append and cached
// attention calls: argument checks and launches.  Included by sdpa_api.cu
// after its helpers.
#pragma once

#include <type_traits>

#include "cache_append.cuh"
#include "paged_attn.cuh"
#include "paged_wide.cuh"
#include "qk_norm_rope.cuh"

namespace {

// A [B][S][H][D] tensor as the checks see it: bytes from its base.
struct View {
    const void* base;
    Strides st;
    int B, S, H, D, elem_bytes;
    long long span() const { return span_bytes(st, B, S, H, D, elem_bytes); }
};

bool view_ok(const View& v)
{
    return strides_ok(v.st, v.elem_bytes) && v.span() >= 0;
}

// Bytes that a view covers, taken modulo `mod` bytes: from its base, the
// reach of the dimensions whose strides are no multiples of mod.
long long extent_modulo(const View& v, long long mod)
{
    const long long st[3] = {v.st.b, v.st.s, v.st.h}, n[3] = {v.B, v.S, v.H};
    __int128 e = v.D;
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && st[i] * v.elem_bytes % mod)
            e += static_cast<__int128>(n[i] - 1) * st[i];
    e *= v.elem_bytes;
    return e > mod ? mod + 1 : static_cast<long long>(e);
}

// True if the two views share no element.  Views whose spans are apart share
// none; neither do two whose addresses lie apart modulo a stride (queries and
// keys in the rows of a fused projection, keys and values side by side in a
// slot of a cache).
bool disjoint(const View& a, const View& b)
{
    if (!overlaps(a.base, a.span(), b.base, b.span()))
        return true;
    const long long strides[3] = {a.st.s, a.st.h, a.st.b};
    for (long long s : strides) {
        const long long mod = s * a.elem_bytes;
        const long long ea = extent_modulo(a, mod), eb = extent_modulo(b, mod);
        long long off = static_cast<long long>(reinterpret_cast<uintptr_t>(b.base) - reinterpret_cast<uintptr_t>(a.base)) % mod;
        if (off < 0)
            off += mod;
        if (off >= ea && off + eb <= mod)
            return true;
    }
    return false;
}

bool same_view(const View& a, const View& b)
{
    return a.base == b.base && a.st.b == b.st.b && a.st.s == b.st.s && a.st.h == b.st.h;
}

// A contiguous buffer of the checks (null: absent).
struct Flat {
    const void* p;
    long long n;
};

bool disjoint_bytes(const View& a, const Flat& f)
{
    return !f.p || !overlaps(a.base, a.span(), f.p, f.n);
}

// The rotation arguments of a call: a table of n_pos rows of rot / 2 pairs.
sdpa_status_t check_rope(const sdpa_rope_t* r, int D)
{
    if (!r || !r->table)
        return SDPA_OK;
    if (r->rot_dim < 8 || r->rot_dim > D || r->rot_dim % 8 != 0)
        return SDPA_ERR_HEAD_DIM;
    if (r->n_pos < 1)
        return SDPA_ERR_BAD_SHAPE;
    if (!aligned16(r->table))
        return SDPA_ERR_MISALIGNED;
    return SDPA_OK;
}

Flat rope_flat(const sdpa_rope_t* r)
{
    if (!r || !r->table)
        return {nullptr, 0};
    return {r->table, static_cast<long long>(r->n_pos) * r->rot_dim * 4};
}

struct NormRopeArgs {
    const void* x[2];
    const void* g[2];
    void* y[2];
    const sdpa_layout_t *xl[2], *gl[2], *yl[2];
    const void* w[2];
    float* dw[2];
    int B, S, H[2], D;
    int norm;
    float eps;
    sdpa_dtype_t dtype, w_dtype;
    const int* positions;
    const sdpa_rope_t* rope;
    void* ws;
    size_t ws_bytes;
    bool backward;
};

// Blocks of each side of the backward pass: shares of rope::kBwdBlocks by the
// side's items, at most one block for each group-sized set of items.
void bwd_blocks(long long tokens, const int* H, int D, int* blocks)
{
    const long long groups = sdpa::rope::kBwdThreads / (D / 8);
    long long items[2], total = 0;
    for (int k = 0; k < 2; ++k) {
        items[k] = tokens * ((H[k] + sdpa::rope::kBwdHeads - 1) / sdpa::rope::kBwdHeads);
        total += items[k];
    }
    for (int k = 0; k < 2; ++k) {
        const long long want = (items[k] + groups - 1) / groups;
        long long share = static_cast<long long>(static_cast<double>(items[k]) / total * sdpa::rope::kBwdBlocks);
        share = share < 1 ? 1 : share;
        blocks[k] = static_cast<int>(items[k] == 0 ? 0 : want < share ? want : share);
    }
}

size_t norm_rope_bwd_workspace(int B, int S, int Hq, int Hkv, int D)
{
    const int H[2] = {Hq, Hkv};
    int blocks[2];
    bwd_blocks(static_cast<long long>(B) * S, H, D, blocks);
    return static_cast<size_t>(blocks[0] + blocks[1]) * D * sizeof(float);
}

template <int D, bool kBF16, bool kInter>
cudaError_t launch_norm_rope(const sdpa::rope::NormRopeParams& p, bool backward, cudaStream_t stream)
{
    using namespace sdpa::rope;
    constexpr int kGroups = kNormThreads / (D / 8);
    if (!backward) {
        const long long items = static_cast<long long>(p.tokens) * (p.side[0].chunks + p.side[1].chunks);
        return launch_pdl(true, norm_rope_kernel<D, kBF16, kInter>, dim3(static_cast<unsigned>((items + kGroups - 1) / kGroups)),
                          dim3(kNormThreads), 0, stream, p);
    }
    cudaError_t e = launch_pdl(true, norm_rope_bwd_kernel<D, kBF16, kInter>, dim3(p.blocks[0] + p.blocks[1]),
                               dim3(kBwdThreads), 0, stream, p);
    if (e == cudaSuccess && p.part)
        e = launch_pdl(true, norm_dw_kernel, dim3(D / kDwCols, p.side[1].H ? 2 : 1), dim3(kDwThreads), 0, stream, p, D);
    return e;
}

template <int D>
cudaError_t launch_norm_rope_d(const sdpa::rope::NormRopeParams& p, bool bf16, bool inter, bool backward, cudaStream_t s)
{
    if (bf16)
        return inter ? launch_norm_rope<D, true, true>(p, backward, s) : launch_norm_rope<D, true, false>(p, backward, s);
    return inter ? launch_norm_rope<D, false, true>(p, backward, s) : launch_norm_rope<D, false, false>(p, backward, s);
}

sdpa_status_t run_norm_rope(NormRopeArgs& a, void* stream)
{
    if ((a.dtype != SDPA_DTYPE_BF16 && a.dtype != SDPA_DTYPE_FP16) ||
        (a.w_dtype != a.dtype && a.w_dtype != SDPA_DTYPE_F32))
        return SDPA_ERR_DTYPE;
    // keys are optional: Hkv = 0 with null pointers
    if (a.B < 1 || a.S < 1 || a.H[0] < 1 || a.H[1] < 0 || (a.H[1] == 0 && (a.x[1] || a.y[1])))
        return SDPA_ERR_BAD_SHAPE;
    const int sides = a.H[1] ? 2 : 1;
    for (int k = 0; k < sides; ++k) {
        if (!a.x[k] || !a.y[k] || (a.backward && !a.g[k]))
            return SDPA_ERR_NULL_PTR;
        if (!aligned16(a.x[k]) || !aligned16(a.y[k]) || !aligned16(a.g[k]) || !aligned(a.w[k], 4) || !aligned(a.dw[k], 4))
            return SDPA_ERR_MISALIGNED;
    }
    if (!aligned(a.positions, 4))
        return SDPA_ERR_MISALIGNED;
    if (a.D != 32 && a.D != 64 && a.D != 128)
        return SDPA_ERR_HEAD_DIM;
    sdpa_status_t st = check_rope(a.rope, a.D);
    if (st != SDPA_OK)
        return st;
    if (a.norm && !(std::isfinite(a.eps) && a.eps >= 0.f))
        return SDPA_ERR_SCALE;
    const long long tokens = static_cast<long long>(a.B) * a.S;
    // items and blocks are counted in 31 bits
    if (tokens > INT32_MAX / 2 ||
        tokens * ((static_cast<long long>(a.H[0]) + a.H[1] + 8) / 4) > INT32_MAX / 2)
        return SDPA_ERR_BAD_SHAPE;
    View x[2], g[2], y[2];
    for (int k = 0; k < sides; ++k) {
        x[k] = View{a.x[k], resolve(a.xl[k], a.S, a.H[k], a.D), a.B, a.S, a.H[k], a.D, 2};
        g[k] = View{a.g[k], resolve(a.gl[k], a.S, a.H[k], a.D), a.B, a.S, a.H[k], a.D, 2};
        y[k] = View{a.y[k], resolve(a.yl[k], a.S, a.H[k], a.D), a.B, a.S, a.H[k], a.D, 2};
        if (!view_ok(x[k]) || !view_ok(y[k]) || (a.backward && !view_ok(g[k])) ||
            !injective(y[k].st, a.B, a.S, a.H[k], a.D))
            return SDPA_ERR_LAYOUT;
    }
    size_t need = 0;
    if (a.backward && a.norm) {
        need = norm_rope_bwd_workspace(a.B, a.S, a.H[0], a.H[1], a.D);
        if (!a.ws)
            return SDPA_ERR_NULL_PTR;
        if (!aligned16(a.ws) || a.ws_bytes < need)
            return SDPA_ERR_WORKSPACE;
    }
    // what is written lies apart from everything else; the forward pass may
    // write a tensor over itself (each row is read before it is written, by
    // the same lanes)
    const int w_bytes = a.w_dtype == SDPA_DTYPE_F32 ? 4 : 2;
    const Flat reads[] = {{a.w[0], a.D * w_bytes}, {a.w[1], a.D * w_bytes}, {a.positions, tokens * 4}, rope_flat(a.rope)};
    const Flat writes[] = {{a.dw[0], a.D * 4}, {a.dw[1], a.D * 4}, {need ? a.ws : nullptr, static_cast<long long>(need)}};
    for (int k = 0; k < sides; ++k) {
        for (int j = 0; j < sides; ++j) {
            if (j != k && !disjoint(y[k], y[j]))
                return SDPA_ERR_ALIAS;
            if (!disjoint(y[k], x[j]) && (a.backward || j != k || !same_view(y[k], x[j])))
                return SDPA_ERR_ALIAS;
            if (a.backward && !disjoint(y[k], g[j]))
                return SDPA_ERR_ALIAS;
        }
        for (const Flat& f : reads)
            if (!disjoint_bytes(y[k], f))
                return SDPA_ERR_ALIAS;
        for (const Flat& f : writes)
            if (!disjoint_bytes(y[k], f) || !disjoint_bytes(x[k], f) || (a.backward && !disjoint_bytes(g[k], f)))
                return SDPA_ERR_ALIAS;
    }
    for (int i = 0; i < 3; ++i) {
        if (!writes[i].p)
            continue;
        for (const Flat& f : reads)
            if (f.p && overlaps(writes[i].p, writes[i].n, f.p, f.n))
                return SDPA_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (writes[j].p && overlaps(writes[i].p, writes[i].n, writes[j].p, writes[j].n))
                return SDPA_ERR_ALIAS;
    }

    int dev = 0, sm_count = 0;
    st = device_ready(&dev, &sm_count);
    if (st != SDPA_OK)
        return st;
    sdpa::rope::NormRopeParams p{};
    const int heads = a.backward ? sdpa::rope::kBwdHeads : sdpa::rope::kHeads;
    for (int k = 0; k < sides; ++k) {
        sdpa::rope::Side& s = p.side[k];
        s.x = a.x[k];
        s.g = a.g[k];
        s.y = a.y[k];
        s.w = a.w[k];
        s.x_sb = x[k].st.b, s.x_ss = x[k].st.s, s.x_sh = x[k].st.h;
        s.g_sb = g[k].st.b, s.g_ss = g[k].st.s, s.g_sh = g[k].st.h;
        s.y_sb = y[k].st.b, s.y_ss = y[k].st.s, s.y_sh = y[k].st.h;
        s.H = a.H[k];
        s.chunks = (a.H[k] + heads - 1) / heads;
        p.dw[k] = a.dw[k];
    }
    if (a.rope && a.rope->table) {
        p.table = a.rope->table;
        p.n_pos = a.rope->n_pos;
        p.rot = a.rope->rot_dim;
    }
    p.positions = a.positions;
    p.S = a.S;
    p.tokens = static_cast<uint32_t>(tokens);
    p.norm = a.norm != 0;
    p.w16 = a.w_dtype != SDPA_DTYPE_F32;
    p.eps = a.eps;
    if (a.backward) {
        bwd_blocks(tokens, a.H, a.D, p.blocks);
        p.part = need ? static_cast<float*>(a.ws) : nullptr;
    }
    const bool bf16 = a.dtype == SDPA_DTYPE_BF16, inter = a.rope && a.rope->table && a.rope->interleaved;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const cudaError_t e = a.D == 32   ? launch_norm_rope_d<32>(p, bf16, inter, a.backward, cs)
                          : a.D == 64 ? launch_norm_rope_d<64>(p, bf16, inter, a.backward, cs)
                                      : launch_norm_rope_d<128>(p, bf16, inter, a.backward, cs);
    return e == cudaSuccess ? SDPA_OK : cuda_fail(e);
}

// Checks of a cache against the shape of a call.
sdpa_status_t check_cache(const sdpa_cache_t* c, const int* table, const int* start, const int* count, int B, int Hkv,
                          int D, int max_pages, View* k, View* v)
{
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !table || !start)
        return SDPA_ERR_NULL_PTR;
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) || !aligned(table, 4) ||
        !aligned(start, 4) || !aligned(count, 4))
        return SDPA_ERR_MISALIGNED;
    if (B < 1 || Hkv < 1 || c->n_pages < 1 || max_pages < 1)
        return SDPA_ERR_BAD_SHAPE;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return SDPA_ERR_BAD_SHAPE;
    if (static_cast<long long>(max_pages) * c->page_size > 1ll << 30)
        return SDPA_ERR_BAD_SHAPE;
    if (D != 64 && D != 128)
        return SDPA_ERR_HEAD_DIM;
    *k = View{c->k, resolve(c->k_layout, c->page_size, Hkv, D), c->n_pages, c->page_size, Hkv, D, 1};
    *v = View{c->v, resolve(c->v_layout, c->page_size, Hkv, D), c->n_pages, c->page_size, Hkv, D, 1};
    if (!view_ok(*k) || !view_ok(*v))
        return SDPA_ERR_LAYOUT;
    return SDPA_OK;
}

sdpa::cache::Pool pool_of(void* codes, float* scale, const View& v)
{
    return {static_cast<uint8_t*>(codes), scale, v.st.b, v.st.s, v.st.h};
}

template <int D, bool kBF16, bool kInter>
cudaError_t launch_append(const sdpa::cache::AppendParams& p, cudaStream_t stream)
{
    using namespace sdpa::cache;
    const long long units = static_cast<long long>(p.B) * p.n_ord * 2 * p.Hkv;
    // one warp a unit holds 4 rows for each of its 256 / D lane groups
    if (p.S <= 4 * (256 / D))
        return launch_pdl(true, append_kernel<D, kBF16, kInter, 1, 4>, dim3(static_cast<unsigned>((units + 7) / 8)),
                          dim3(kAppendThreads), 0, stream, p);
    // eight warps a unit: 2048 / D rows a pass, as many passes as a page has
    auto go = [&](auto passes) {
        return launch_pdl(true, append_kernel<D, kBF16, kInter, 8, decltype(passes)::value>, dim3(static_cast<unsigned>(units)),
                          dim3(kAppendThreads), 0, stream, p);
    };
    const int passes = (p.page * D + 2047) / 2048;
    if (passes <= 1)
        return go(std::integral_constant<int, 1>{});
    if (passes <= 2)
        return go(std::integral_constant<int, 2>{});
    if (passes <= 4)
        return go(std::integral_constant<int, 4>{});
    return go(std::integral_constant<int, 8>{});
}

template <int D>
cudaError_t launch_append_d(const sdpa::cache::AppendParams& p, bool bf16, bool inter, cudaStream_t s)
{
    if (bf16)
        return inter ? launch_append<D, true, true>(p, s) : launch_append<D, true, false>(p, s);
    return inter ? launch_append<D, false, true>(p, s) : launch_append<D, false, false>(p, s);
}

// Attention over a paged cache: rows of a tile (8, 16, or 128 with the wide
// kernel), and the CTAs that share the key tiles (two on each of 152 SMs, one
// of the wide kernel).
constexpr int kPagedCtas = 304;

int paged_tile_rows(int Sq, int group)
{
    const long long rows = static_cast<long long>(Sq) * group;
    return rows <= 8 ? 8 : rows <= 16 ? 16 : sdpa::paged::kWideRows;
}

int paged_ctas(int tile_rows)
{
    return tile_rows == sdpa::paged::kWideRows ? kPagedCtas / 2 : kPagedCtas;
}

// The pieces' results, their LSE, and what is to join.
size_t paged_workspace(int Hq, int Hkv, int Sq, int D)
{
    const int nr = paged_tile_rows(Sq, Hq / Hkv);
    return static_cast<size_t>(paged_ctas(nr)) * (2 * nr * (D + 1) * sizeof(float) + sizeof(int4));
}

template <int D, bool kBF16, int NR>
cudaError_t launch_paged(const CUtensorMap& tk, const CUtensorMap& tv, const sdpa::paged::Params& p, int dev,
                         cudaStream_t stream)
{
    using namespace sdpa::paged;
    static std::once_flag once[kMaxDevices];
    static cudaError_t attr[kMaxDevices];
    constexpr bool kWide = NR == kWideRows;
    auto* kernel = [] {
        if constexpr (kWide)
            return paged_wide_kernel<D, kBF16>;
        else
            return paged_attn_kernel<D, kBF16, NR>;
    }();
    using L = std::conditional_t<kWide, WideLayout<D, kBF16>, PagedLayout<D, kBF16, kWide ? 16 : NR>>;
    std::call_once(once[dev], [&] {
        attr[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmemBytes);
    });
    if (attr[dev] != cudaSuccess)
        return attr[dev];
    cudaError_t e = launch_pdl(true, kernel, dim3(p.ctas), dim3(L::kThreads), L::kSmemBytes, stream, tk, tv, p);
    const long long rows = static_cast<long long>(p.Sq) * p.group;
    const unsigned blocks = static_cast<unsigned>(kWide ? (rows < NR ? rows + 7 : NR) / 8 : rows < NR ? rows : NR);
    if (e == cudaSuccess && p.ctas > 1)
        e = launch_pdl(true, paged_join_kernel<D, kBF16, NR>, dim3(p.ctas - 1, blocks), dim3(kJoinThreads), 0, stream, p);
    return e;
}

template <int D, bool kBF16>
cudaError_t launch_paged_rows(int nr, const CUtensorMap& tk, const CUtensorMap& tv, const sdpa::paged::Params& p, int dev,
                              cudaStream_t s)
{
    return nr == 8    ? launch_paged<D, kBF16, 8>(tk, tv, p, dev, s)
           : nr == 16 ? launch_paged<D, kBF16, 16>(tk, tv, p, dev, s)
                      : launch_paged<D, kBF16, sdpa::paged::kWideRows>(tk, tv, p, dev, s);
}

}  // namespace

extern "C" {

sdpa_status_t sdpa_qk_norm_rope(const void* Q, const void* K, void* Q_out, void* K_out, int B, int S, int Hq, int Hkv,
                                int D, const sdpa_layout_t* q_layout, const sdpa_layout_t* k_layout,
                                const sdpa_layout_t* q_out_layout, const sdpa_layout_t* k_out_layout, int norm,
                                const void* q_weight, const void* k_weight, sdpa_dtype_t weight_dtype, float eps,
                                const sdpa_rope_t* rope, const int* positions, sdpa_dtype_t dtype, void* stream)
{
    NormRopeArgs a{{Q, K}, {nullptr, nullptr}, {Q_out, K_out}, {q_layout, k_layout}, {nullptr, nullptr},
                   {q_out_layout, k_out_layout}, {q_weight, k_weight}, {nullptr, nullptr}, B, S, {Hq, Hkv}, D, norm, eps,
                   dtype, weight_dtype, positions, rope, nullptr, 0, false};
    return run_norm_rope(a, stream);
}

sdpa_status_t sdpa_qk_norm_rope_bwd(const void* Q, const void* K, const void* dQ_out, const void* dK_out, void* dQ,
                                    void* dK, float* dq_weight, float* dk_weight, int B, int S, int Hq, int Hkv, int D,
                                    const sdpa_layout_t* q_layout, const sdpa_layout_t* k_layout,
                                    const sdpa_layout_t* dq_out_layout, const sdpa_layout_t* dk_out_layout,
                                    const sdpa_layout_t* dq_layout, const sdpa_layout_t* dk_layout, int norm,
                                    const void* q_weight, const void* k_weight, sdpa_dtype_t weight_dtype, float eps,
                                    const sdpa_rope_t* rope, const int* positions, sdpa_dtype_t dtype, void* workspace,
                                    size_t workspace_bytes, void* stream)
{
    NormRopeArgs a{{Q, K}, {dQ_out, dK_out}, {dQ, dK}, {q_layout, k_layout}, {dq_out_layout, dk_out_layout},
                   {dq_layout, dk_layout}, {q_weight, k_weight}, {dq_weight, dk_weight}, B, S, {Hq, Hkv}, D, norm, eps,
                   dtype, weight_dtype, positions, rope, workspace, workspace_bytes, true};
    return run_norm_rope(a, stream);
}

size_t sdpa_qk_norm_rope_bwd_workspace_bytes(int B, int S, int Hq, int Hkv, int D)
{
    if (B < 1 || S < 1 || Hq < 1 || Hkv < 0 || (D != 32 && D != 64 && D != 128))
        return 0;
    return norm_rope_bwd_workspace(B, S, Hq, Hkv, D);
}

sdpa_status_t sdpa_cache_append(const void* K, const void* V, const sdpa_cache_t* cache, const int* block_table,
                                const int* start, const int* count, int B, int S, int Hkv, int D, int max_pages,
                                const sdpa_layout_t* k_layout, const sdpa_layout_t* v_layout, const sdpa_rope_t* rope,
                                sdpa_dtype_t dtype, void* stream)
{
    if (dtype != SDPA_DTYPE_BF16 && dtype != SDPA_DTYPE_FP16)
        return SDPA_ERR_DTYPE;
    if (!K || !V)
        return SDPA_ERR_NULL_PTR;
    if (!aligned16(K) || !aligned16(V))
        return SDPA_ERR_MISALIGNED;
    View ck, cv;
    sdpa_status_t st = check_cache(cache, block_table, start, count, B, Hkv, D, max_pages, &ck, &cv);
    if (st != SDPA_OK)
        return st;
    if (S < 1)
        return SDPA_ERR_BAD_SHAPE;
    st = check_rope(rope, D);
    if (st != SDPA_OK)
        return st;
    const View k{K, resolve(k_layout, S, Hkv, D), B, S, Hkv, D, 2}, v{V, resolve(v_layout, S, Hkv, D), B, S, Hkv, D, 2};
    if (!view_ok(k) || !view_ok(v) || !injective(ck.st, ck.B, ck.S, Hkv, D) || !injective(cv.st, cv.B, cv.S, Hkv, D))
        return SDPA_ERR_LAYOUT;
    const int page = cache->page_size;
    const int n_ord = static_cast<int>((static_cast<long long>(S) + page - 2) / page + 1);
    if (static_cast<__int128>(B) * n_ord * 2 * Hkv > INT32_MAX)
        return SDPA_ERR_BAD_SHAPE;
    // the codes and scales lie apart from one another and from what is read
    const long long sc = static_cast<long long>(cache->n_pages) * Hkv * 4;
    const View* codes[2] = {&ck, &cv};
    const Flat flat[] = {{cache->k_scale, sc}, {cache->v_scale, sc}, {block_table, 4ll * B * max_pages}, {start, 4ll * B},
                         {count, 4ll * B}, rope_flat(rope)};
    if (!disjoint(ck, cv) || overlaps(cache->k_scale, sc, cache->v_scale, sc))
        return SDPA_ERR_ALIAS;
    for (int i = 0; i < 2; ++i) {
        if (!disjoint(*codes[i], k) || !disjoint(*codes[i], v) || !disjoint_bytes(k, flat[i]) || !disjoint_bytes(v, flat[i]))
            return SDPA_ERR_ALIAS;
        for (int j = 0; j < 6; ++j)
            if (!disjoint_bytes(*codes[i], flat[j]) ||
                (j > 1 && flat[j].p && overlaps(flat[i].p, flat[i].n, flat[j].p, flat[j].n)))
                return SDPA_ERR_ALIAS;
    }

    int dev = 0, sm_count = 0;
    st = device_ready(&dev, &sm_count);
    if (st != SDPA_OK)
        return st;
    sdpa::cache::AppendParams p{};
    p.x[0] = K;
    p.x[1] = V;
    p.x_sb[0] = k.st.b, p.x_ss[0] = k.st.s, p.x_sh[0] = k.st.h;
    p.x_sb[1] = v.st.b, p.x_ss[1] = v.st.s, p.x_sh[1] = v.st.h;
    p.pool[0] = pool_of(cache->k, cache->k_scale, ck);
    p.pool[1] = pool_of(cache->v, cache->v_scale, cv);
    p.table = block_table;
    p.start = start;
    p.count = count;
    p.B = B;
    p.S = S;
    p.Hkv = Hkv;
    p.page = page;
    p.page_shift = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
    p.n_pages = cache->n_pages;
    p.max_pages = max_pages;
    p.n_ord = n_ord;
    bool inter = false;
    if (rope && rope->table) {
        p.rope = rope->table;
        p.n_pos = rope->n_pos;
        p.rot = rope->rot_dim;
        inter = rope->interleaved != 0;
    }
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == SDPA_DTYPE_BF16;
    const cudaError_t e = D == 64 ? launch_append_d<64>(p, bf16, inter, cs) : launch_append_d<128>(p, bf16, inter, cs);
    return e == cudaSuccess ? SDPA_OK : cuda_fail(e);
}

sdpa_status_t sdpa_fwd_paged(const void* Q, const sdpa_cache_t* cache, const int* block_table, const int* start,
                             const int* count, void* O, float* LSE, int B, int Hq, int Hkv, int Sq, int D, int max_pages,
                             const sdpa_layout_t* q_layout, const sdpa_layout_t* o_layout, float scale, int causal,
                             sdpa_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream)
{
    if (dtype != SDPA_DTYPE_BF16 && dtype != SDPA_DTYPE_FP16)
        return SDPA_ERR_DTYPE;
    if (!Q || !O)
        return SDPA_ERR_NULL_PTR;
    if (!aligned16(Q) || !aligned16(O) || !aligned(LSE, 4))
        return SDPA_ERR_MISALIGNED;
    View ck, cv;
    sdpa_status_t st = check_cache(cache, block_table, start, count, B, Hkv, D, max_pages, &ck, &cv);
    if (st != SDPA_OK)
        return st;
    if (Sq < 1 || Hq < 1)
        return SDPA_ERR_BAD_SHAPE;
    if (Hq % Hkv != 0)
        return SDPA_ERR_HEADS;
    if (static_cast<__int128>(B) * Sq * Hq > INT32_MAX)
        return SDPA_ERR_BAD_SHAPE;
    // (the kernels' factor, with log2(e), has to be finite as well)
    const float scale_log2 = static_cast<float>(scale * 1.4426950408889634);
    if (!valid_scale(scale) || !std::isfinite(scale_log2))
        return SDPA_ERR_SCALE;
    const View q{Q, resolve(q_layout, Sq, Hq, D), B, Sq, Hq, D, 2}, o{O, resolve(o_layout, Sq, Hq, D), B, Sq, Hq, D, 2};
    if (!view_ok(q) || !view_ok(o) || !injective(o.st, B, Sq, Hq, D))
        return SDPA_ERR_LAYOUT;
    const size_t need = paged_workspace(Hq, Hkv, Sq, D);
    if (!workspace)
        return SDPA_ERR_NULL_PTR;
    if (!aligned16(workspace) || workspace_bytes < need)
        return SDPA_ERR_WORKSPACE;
    // O, LSE and the workspace lie apart from one another and from every input
    const long long sc = static_cast<long long>(cache->n_pages) * Hkv * 4;
    const long long lse_bytes = LSE ? static_cast<long long>(B) * Hq * Sq * 4 : 0;
    const Flat flat[] = {{cache->k, ck.span()}, {cache->v, cv.span()}, {cache->k_scale, sc}, {cache->v_scale, sc},
                         {block_table, 4ll * B * max_pages}, {start, 4ll * B}, {count, 4ll * B}, {Q, q.span()},
                         {O, o.span()}, {LSE, lse_bytes}, {workspace, static_cast<long long>(need)}};
    constexpr int kQ = 7, kO = 8, kAll = 11;         // flat[8..10] are written
    for (int w = kO; w < kAll; ++w)
        for (int i = 0; i < w; ++i)
            if (flat[w].p && flat[i].p && overlaps(flat[w].p, flat[w].n, flat[i].p, flat[i].n) &&
                !(w == kO && i == kQ && disjoint(o, q)))
                return SDPA_ERR_ALIAS;

    int dev = 0, sm_count = 0;
    st = device_ready(&dev, &sm_count);
    if (st != SDPA_OK)
        return st;
    sdpa::paged::Params p{};
    p.Q = Q;
    p.O = O;
    p.lse = LSE;
    p.q_sb = q.st.b, p.q_ss = q.st.s, p.q_sh = q.st.h;
    p.o_sb = o.st.b, p.o_ss = o.st.s, p.o_sh = o.st.h;
    p.k = pool_of(cache->k, cache->k_scale, ck);
    p.v = pool_of(cache->v, cache->v_scale, cv);
    p.table = block_table;
    p.start = start;
    p.count = count;
    p.B = B;
    p.Sq = Sq;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.group = Hq / Hkv;
    p.page = cache->page_size;
    p.n_pages = cache->n_pages;
    p.max_pages = max_pages;
    p.causal = causal ? 1 : 0;
    p.scale_log2 = scale_log2;
    p.page_shift = p.page == 16 ? 4 : p.page == 32 ? 5 : p.page == 64 ? 6 : 7;
    const int nr = paged_tile_rows(Sq, p.group);
    p.row_tiles = static_cast<int>((static_cast<long long>(Sq) * p.group + nr - 1) / nr);
    // no more CTAs than there can be tiles
    const __int128 most = static_cast<__int128>(B) * Hkv * p.row_tiles *
                          ((static_cast<long long>(max_pages) * p.page + sdpa::paged::kTileKeys - 1) / sdpa::paged::kTileKeys);
    const int per_sm = nr == sdpa::paged::kWideRows ? 1 : 2;
    p.ctas = per_sm * sm_count < paged_ctas(nr) ? per_sm * sm_count : paged_ctas(nr);
    p.ctas = most < p.ctas ? static_cast<int>(most) : p.ctas;
    p.part_o = static_cast<float*>(workspace);
    p.ctas_inverse = ~0ull / p.ctas + 1;
    p.part_lse = p.part_o + static_cast<long long>(p.ctas) * 2 * nr * D;
    p.joins = reinterpret_cast<int4*>(p.part_lse + static_cast<long long>(p.ctas) * 2 * nr);
    // L2 fetches no more than a slot's bytes where the slots of a head lie
    // apart: 256-byte fetches would bring in the neighbour head's half each
    // time
    auto map = [&](CUtensorMap* m, const void* base, const Strides& st) {
        return make_map(m, base, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, D, Hkv, p.page, p.n_pages, st, 1, p.page,
                        st.s == D    ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                        : D == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                   : CU_TENSOR_MAP_L2_PROMOTION_L2_64B);
    };
    CUtensorMap tk, tv;
    if (!map(&tk, cache->k, ck.st) || !map(&tv, cache->v, cv.st))
        return cuda_fail(cudaErrorInvalidValue);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == SDPA_DTYPE_BF16;
    const cudaError_t e = D == 64 ? (bf16 ? launch_paged_rows<64, true>(nr, tk, tv, p, dev, cs)
                                          : launch_paged_rows<64, false>(nr, tk, tv, p, dev, cs))
                                  : (bf16 ? launch_paged_rows<128, true>(nr, tk, tv, p, dev, cs)
                                          : launch_paged_rows<128, false>(nr, tk, tv, p, dev, cs));
    return e == cudaSuccess ? SDPA_OK : cuda_fail(e);
}

size_t sdpa_paged_workspace_bytes(int B, int Hq, int Hkv, int Sq, int D)
{
    if (B < 1 || Hq < 1 || Hkv < 1 || Sq < 1 || Hq % Hkv != 0 || (D != 64 && D != 128))
        return 0;
    return paged_workspace(Hq, Hkv, Sq, D);
}

}  // extern "C"
