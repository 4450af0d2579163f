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

// Sequences of an attention call, at most.
constexpr int kMaxSeqs = 1024;

// Attention over a cache: CTAs of the kernel for few rows, and whether it takes a
// call: sequences of at most 32 rows (tokens x heads of a group) on average. (Groups
// of 8, 4 heads; this kernel or the one on tiles with 16, 32 and 64 rows. Heads of 128:
// 64 sequences of 16,384 keys 187 or 470 us, 326 or 468, 611 or 644; 8 of them 50 or 75,
// 77 or 75, 128 or 76; 8 of 1,024 keys 18 or 26, 33 or 26, 35 or 27. Heads of 64: 8 of
// 16,384 keys 31 or 58, 43 or 59, 68 or 60. So at 32 rows the rule is right for many
// sequences or heads of 64, and up to 27% off for few of 128: their number is not in it.)
constexpr int kAttendSms = 152;
inline bool attend_few(long long rows, int group, int seqs) { return group <= 16 && rows * group <= 32LL * seqs; }
// Rows of its tiles, at most: 8 where the group has no more heads and the call
// about one token for each sequence, or as few as 8 tiles of 8. (Two tokens of groups
// of 8, 4 heads of 128, tiles of 8 or 16: one sequence of 16,384 19 or 26 us, 8 of them
// 56 or 51, 64 of them 224 or 195.)
inline int attend_few_rows(long long rows, int group, int seqs, int heads) {
  return group <= 8 && (rows * group <= 8LL * seqs || rows * group * heads <= 64) ? 8 : 16;
}
// Whether each warp takes a piece of the work for itself (16, or with tiles of 16
// rows 12, on an SM), or each SM: with many tiles. (8,191 keys of 128 elements, groups
// of 4, warps or SMs: 256 tiles 77 or 96 us, 128 tiles 57 or 57, 64 tiles 66 or 41;
// 1,023 keys: 32 or 39, 33 or 26, 38 or 14.)
inline bool attend_few_alone(int seqs, int heads) { return 4LL * seqs * heads >= 5 * kAttendSms; }
constexpr int attend_few_pieces(int rows, bool alone) { return kAttendSms * (alone ? (rows == 8 ? 16 : 12) : 1); }

// The kernel on tensor-core tiles: items (pairs of tiles of 128 rows) that are at most
// half as many as the SMs are cut into pieces, no more than SMs.
constexpr int kAttendMaxPieces = kAttendSms;
// Whether a call may have so few items: if even all its rows side by side make
// fewer. (Rows of no sequence may leave fewer than counted here; those calls are not
// cut.)
inline bool attend_may_cut(long long rows, int group, int heads) {
  const long long pair = 2 * (128 / group);
  return 2 * ((rows + pair - 1) / pair * heads) <= kAttendSms;
}

}  // namespace plan
}  // namespace clover
