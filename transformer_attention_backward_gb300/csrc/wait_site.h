// Where a device-side wait ran out, as one word: written by the kernel that
// gives up first, read by abw_device_check.  Plain C++, for both sides.
#pragma once

namespace abw {

enum : unsigned int {
  kSiteKv = 1u, kSiteDq, kSiteFwd, kSiteDecode, kSiteLinState, kSiteLinOut, kSiteLinGrad, kSiteEnd,
  kSiteWinFwd = kSiteEnd, kSiteWinKv, kSiteWinDq, kSiteWinEnd   // the windowed attention's
};

struct WaitSite {
  unsigned int kernel, slot, warp, block;
};

// Kernel in bits 28-31, barrier slot in bits 21-27, warp of the block (up to 32
// of them) in bits 16-20, and the low 16 bits of the block index.
constexpr unsigned int pack_site(const WaitSite &s) {
  return (s.kernel << 28) | ((s.slot & 0x7fu) << 21) | ((s.warp & 0x1fu) << 16) | (s.block & 0xffffu);
}
constexpr WaitSite unpack_site(unsigned int w) {
  return WaitSite{w >> 28, (w >> 21) & 0x7fu, (w >> 16) & 0x1fu, w & 0xffffu};
}
static_assert(kSiteWinEnd <= 16, "four bits for the kernel");

inline const char *site_kernel(unsigned int kernel) {
  switch (kernel) {
    case kSiteKv: return "causal kv";
    case kSiteDq: return "causal dq";
    case kSiteFwd: return "causal forward";
    case kSiteDecode: return "decode";
    case kSiteLinState: return "linear attention state";
    case kSiteLinOut: return "linear attention output";
    case kSiteLinGrad: return "linear attention gradient";
    case kSiteWinFwd: return "window forward";
    case kSiteWinKv: return "window kv";
    case kSiteWinDq: return "window dq";
    default: return "?";
  }
}

}  // namespace abw
