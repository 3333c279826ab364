// page_attn.cu -- attention of each request's new tokens over its pages:
// lbx_paged_attention (host side; the kernel is in page_attn.cuh).
#include "page_attn.cuh"

namespace lbx {
namespace paged {
namespace {

constexpr long long kWideRows = 768;
constexpr size_t kCounterBytes = (kFewUnits * kMaxCtas * 4 + 255) & ~255;
static_assert(kFewUnits >= 2, "counters of two subtiles per CTA, or of the lists of few rows");
// the units' partials of few rows lie where those of tiles do
template <int DH>
constexpr bool kFewFits =
    (size_t)kFewUnits * kMaxCtas * kFewPart<DH> <= (DH == 256 ? 2 : 4) * kMaxCtas * part_floats(DH);
static_assert(kFewFits<64> && kFewFits<128> && kFewFits<256>, "partials");

bool encode_pool(CUtensorMap *map, const void *base, const lbx_page_cfg *c, int box) {
  const uint64_t row = (uint64_t)c->Hkv * c->dh * 2;
  const uint64_t dims[3] = {(uint64_t)c->dh, (uint64_t)c->Hkv,
                            (uint64_t)c->L * c->n_pages * c->page};
  const uint64_t strides[2] = {(uint64_t)c->dh * 2, row};
  const uint32_t boxes[3] = {64, 1, (uint32_t)box};
  return cache::encode_16bit(map, base, 3, dims, strides, boxes);
}

}  // namespace
}  // namespace paged
}  // namespace lbx

extern "C" size_t lbx_paged_workspace_size(const lbx_page_cfg *c) {
  using namespace lbx::paged;
  if (!cfg_ok(c) || c->Hq / c->Hkv > LBX_PAGED_MAX_GROUP) return 0;
  // per CTA a tile's first piece and another one, of each of its subtiles
  const size_t parts = c->dh == 256 ? 2 * kMaxCtas : 4 * kMaxCtas;
  return kCounterBytes + parts * part_floats(c->dh) * 4;
}

extern "C" int lbx_paged_attention(const lbx_page_cfg *c, const int32_t *start,
                                   const int32_t *ctx_len, const int32_t *block_table,
                                   const int32_t *parent, const uint16_t *q,
                                   const uint16_t *k_pages, const uint16_t *v_pages, uint16_t *o,
                                   float *lse, void *workspace, size_t workspace_bytes,
                                   int32_t *d_status, cudaStream_t stream) {
  using namespace lbx::paged;
  const size_t need = lbx_paged_workspace_size(c);
  if (need == 0 || workspace_bytes < need) return LBX_EINVAL;
  for (const int32_t *p : {start, ctx_len, block_table})
    if (!aligned_to(p, 4)) return LBX_EINVAL;
  for (const uint16_t *p : {q, k_pages, v_pages, (const uint16_t *)o})
    if (!aligned_to(p, 16)) return LBX_EINVAL;
  if ((parent && !aligned_to(parent, 4)) || (lse && !aligned_to(lse, 4)) ||
      !aligned_to(workspace, 16) || (d_status && !aligned_to(d_status, 4)))
    return LBX_EINVAL;
  // tiles of one request read q while others write o
  const size_t rows = (size_t)c->L * c->M * c->Hq, values = rows * c->dh * 2;
  if (!all_apart({{o, values}, {lse, lse ? rows * 4 : 0}, {workspace, need}}, {{q, values}}))
    return LBX_EINVAL;
  PageArgs A = {};
  A.c = *c;
  A.G = c->Hq / c->Hkv, A.tp = kRows / A.G, A.box = c->page < 64 ? c->page : 64;
  while (1 << A.shift < c->page) ++A.shift;
  // Head dimension 128: a pair of CTAs shares products of 256 rows of both of its subtiles,
  // which halves what shared memory has to deliver (prompts of 501 to 6001 tokens, 32/8
  // heads: 508 us against 556 us on single CTAs); requests of few rows leave the second
  // subtile empty and are better off with more and smaller tiles (16 requests of one token
  // over 8001 to 16384 keys: 487 us against 845 us).  The lengths are on the device: M and
  // Bq decide, by the rows of a request on average, padding included (it is what the header tells
  // callers: these single tokens padded to 4096 rows take 841 us).  16 requests over 3000 keys, 32/8 heads,
  // pairs against single CTAs: 192 tokens (768 rows) 154 against 135 us, 256 tokens 169
  // against 177 us, 512 tokens 329 against 358 us.
  const bool wide = c->dh == 128 && (long long)c->M * A.G > kWideRows * (long long)c->Bq;
  A.shape = shape_of(A.G, wide ? 4 : 2, parent != nullptr);
  A.scale_log2 = c->scale * 1.4426950408889634f;
  A.start = start, A.ctx_len = ctx_len, A.table = block_table, A.parent = parent;
  A.q = q, A.k = k_pages, A.v = v_pages, A.o = o, A.lse = lse, A.status = d_status;
  A.counters = static_cast<unsigned int *>(workspace);
  A.part = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + kCounterBytes);

  PageMaps maps;
  const uint64_t row = (uint64_t)c->Hq * c->dh * 2;
  const uint64_t dims[4] = {(uint64_t)c->dh, (uint64_t)c->Hq, (uint64_t)c->M, (uint64_t)c->L};
  const uint64_t strides[3] = {(uint64_t)c->dh * 2, row, row * (uint64_t)c->M};
  const uint32_t box[4] = {64, (uint32_t)A.G, (uint32_t)A.tp, 1};
  if (!lbx::cache::encode_16bit(&maps.q, q, 4, dims, strides, box) ||
      !lbx::cache::encode_16bit(&maps.o, o, 4, dims, strides, box) ||
      !encode_pool(&maps.k, k_pages, c, A.box) || !encode_pool(&maps.v, v_pages, c, A.box))
    return LBX_ECUDA;
  const int nsm = lbx::cache::grid_limit();
  if (nsm < 2) return LBX_ECUDA;
  const int grid = nsm / 2 * 2;
  const bool f16 = c->dtype == LBX_F16;
  const bool split = c->weights == LBX_WEIGHTS_SPLIT;
  const auto launch = c->dh == 64    ? split ? launch_page_attn<64, false, true> : launch_page_attn<64, false, false>
                      : c->dh == 256 ? split ? launch_page_attn<256, false, true> : launch_page_attn<256, false, false>
                      : wide         ? split ? launch_page_attn<128, true, true> : launch_page_attn<128, true, false>
                      : split        ? launch_page_attn<128, false, true>
                                     : launch_page_attn<128, false, false>;
  return launch(f16, maps, A, grid, stream) == cudaSuccess ? LBX_OK : LBX_ECUDA;
}
