// Launch planning for the persistent MoE kernels: which kernel takes a call
// and how large its grid is. Plain C++ with no CUDA dependency, so the
// decisions can be checked on a host without a GPU for any SM count.
#pragma once

namespace clover {
namespace plan {

// Largest token count of the fused layer kernel (one 32-bit mask per
// expert) and the most router rows one of its CTAs stages.
constexpr int kFusedMaxTokens = 32;
constexpr int kFusedRouterRowsPerCta = 8;

// The fused layer kernel (routing + experts + combine in one launch) takes a
// call when the tokens fit its masks, every CTA's share of the router rows
// fits its staging slices, and there is one CTA per token for the top-k
// selection (CTA t selects token t).
inline bool moe_fused(int tokens, int experts, int grid) {
  return grid >= 1 && tokens <= kFusedMaxTokens && grid >= tokens &&
         (experts + grid - 1) / grid <= kFusedRouterRowsPerCta;
}

// Grid of a persistent kernel whose CTAs wait on one another at grid
// barriers, so all of them must be resident at once. The kernels are written
// for one CTA per SM; resident_per_sm is what the occupancy query reports for
// the kernel at its shared-memory size. Returns the grid (one CTA per SM), or
// 0 when not even one CTA fits on an SM: such a launch would leave CTAs
// waiting for SMs that a barrier holds, so it is rejected instead.
inline int persistent_grid(int sms, int resident_per_sm) {
  if (sms < 1 || resident_per_sm < 1) return 0;
  return sms;
}

// Whether a grouped 4-bit product runs on pairs of CTAs (tiles of 256 rows)
// rather than single ones (128). A pair takes in fewer bytes per product, but
// waits longer between tiles and fills its tiles worse: it needs long groups
// and a long K (single -> pair on one box: 8,192^3 195 -> 178 us, SwiGLU with N =
// K = 8,192 186 -> 161, with K = 4,096 104 -> 99; but plain with K = 4,096 111 ->
// 114, with K = 2,048 74 -> 83, and 64 groups of about 256 rows 150 -> 174). Not
// timed, and left to single CTAs: a plain K between 4,096 and 8,192, groups between
// 256 and 1,024 rows. N is not asked about: 256 rows of it make a tile either way.
inline bool fp4_pairs(int rows, int groups, int k, bool swiglu) {
  return rows / groups >= 1024 && k >= (swiglu ? 4096 : 8192);
}

// Expert routing: CTAs of 8 warps, one token per warp and round. Up to 64
// tokens one cluster of up to 8 CTAs selects and groups in one launch (64 tokens
// on one box: 5.3 us, as three launches 7.0). Beyond, the tokens spread over
// more CTAs, which leave their counts per expert; a second launch scans them and
// a third places the slots. (Without the second, each CTA of the third adding
// up all counts itself: 257 tokens 11.2 instead of 10.0 us, 1,024 19.8 instead
// of 9.6.)
constexpr int kRouteWarps = 8;
constexpr int kRouteClusterTokens = 64;
constexpr int kRouteCtaTokens = 64;  // at most: one bit each in an expert's token mask
// CTAs that fill the machine (4 on each of 152 SMs). The tokens are spread over
// that many as evenly as 64 per CTA allow: with fewer and larger ones some SMs
// hold four and others none, as a launch fills what the one before it frees
// (32,768 tokens in 512 CTAs of 64: 50 us, in 607 of 54: 45 us).
constexpr int kRouteFullCtas = 608;

struct RouteShape {
  int cta_tokens;  // tokens per CTA
  int ctas;
  bool cluster;    // all of them one cluster
};

// Most CTAs any call of at most this many tokens uses: what a workspace holds.
inline int route_max_ctas(int tokens) {
  const int most = (tokens + kRouteWarps - 1) / kRouteWarps;
  const int full = (tokens + kRouteCtaTokens - 1) / kRouteCtaTokens;
  return full > kRouteFullCtas ? full : (most < kRouteFullCtas ? most : kRouteFullCtas);
}

inline RouteShape route_shape(int tokens) {
  RouteShape s;
  s.cta_tokens = kRouteWarps;
  s.cluster = tokens <= kRouteClusterTokens;
  if (s.cluster) {
    s.ctas = 1;
    while (s.ctas * s.cta_tokens < tokens) s.ctas *= 2;
  } else {
    const int even = (tokens + kRouteFullCtas - 1) / kRouteFullCtas;
    if (even > s.cta_tokens) s.cta_tokens = even < kRouteCtaTokens ? even : kRouteCtaTokens;
    s.ctas = (tokens + s.cta_tokens - 1) / s.cta_tokens;
  }
  return s;
}

}  // namespace plan
}  // namespace clover
