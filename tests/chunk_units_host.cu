// The chunk attention's work-split arithmetic, compiled for the host from its own source, for
// tests/test_chunk_units_host.py.  Reciprocals are off by a chosen number of ulps, as the device's may be.
#include <cmath>

static int g_ulps = 0;
static float host_rcp(float x) {
  float r = 1.f / x;
  for (int i = 0; i < (g_ulps < 0 ? -g_ulps : g_ulps); ++i) r = std::nextafterf(r, g_ulps < 0 ? 0.f : INFINITY);
  return r;
}
#define LLAMA_HOST_RCP(x) host_rcp(x)
#include "chunk_attn.cu"

namespace llama {   // what the launch code refers to; nothing here is launched
bool encode_tmap_3d_bf16(CUtensorMap*, const void*, uint64_t, uint64_t, uint64_t, uint64_t, uint64_t, uint32_t, uint32_t,
                         uint32_t) { return false; }
bool encode_tmap_4d_bf16(CUtensorMap*, const void*, const uint64_t*, const uint64_t*, const uint32_t*) { return false; }
void set_pdl(bool) {}
bool pdl_enabled() { return false; }
}  // namespace llama

extern "C" {
void host_ulps(int n) { g_ulps = n; }
int host_div_by(int a, int b) { return llama::div_by(a, b, llama::rcp((float)b)); }
int host_div_inv(int a, int b) { return llama::div_inv(a, b, llama::inverse(b)); }
int host_candidate(int w) { return llama::candidate(w); }
void host_cut(int nt, int C, int* out) { llama::cut(nt, C, llama::rcp((float)C), out[0], out[1]); }
// seq: unit0, lo, n, c, np, wp, span, nc, ct, cut_n, part0, split0
int host_unit(int r, int n_kv, const int* seq, int u, int* out) {
  llama::ChunkParams p;
  memset(&p, 0, sizeof(p));
  p.n_kv = n_kv;
  p.inv_kv = llama::inverse(n_kv);
  p.tpt = 128 / r;
  llama::ChunkSeq s;
  static_assert(sizeof(s) == 12 * sizeof(int), "the sequence's record");
  memcpy(&s, seq, sizeof(s));
  llama::ChunkUnit d;
  memset(&d, 0, sizeof(d));
  const bool live = llama::make_unit(p, s, 0, u, d);
  const int v[] = {d.g, d.t0, d.n0, d.n1, d.lone, d.row0, d.row1, d.part, d.end, d.pos_off, d.kv_len, d.clean};
  memcpy(out, v, sizeof(v));
  return live;
}
}
