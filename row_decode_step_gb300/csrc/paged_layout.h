// How dl_paged_attn divides its workspace (host arithmetic only): the counters, then the parts.
//
// One workspace serves calls of every tile size and, where it is large enough, of either head width.  The
// instances differ in CTAs and in a part's size, but not in where the parts begin: no call may leave anything in
// the counters of another, which are zero between calls.
#pragma once

#include <cstddef>

namespace dlp {

// CTAs of an instance (head width D, tiles of QT queries) that an SM holds (registers: at most 128 or 168 a
// thread).  For QT = 4 and D = 128, four CTAs of 128 registers spill and were slower (64 ragged sequences
// 57 us against 52).
constexpr int attn_ctas_per_sm(int D, int QT) { return D == 64 && QT == 4 ? 4 : 3; }
constexpr int kMostCtasPerSm = 4;

struct AttnLayout {
    int grid;                                // the most CTAs of a call
    size_t counters, parts;                  // bytes, one after the other
    size_t total() const { return counters + parts; }
};

// Three counters a CTA; two parts a CTA, each of QT x (D + 2) floats.
inline AttnLayout attn_layout(int sms, int D, int QT)
{
    AttnLayout l;
    l.grid = sms * attn_ctas_per_sm(D, QT);
    l.counters = (size_t)sms * kMostCtasPerSm * 3 * 4;
    l.counters = (l.counters + 15) / 16 * 16;
    l.parts = (size_t)l.grid * 2 * QT * (D + 2) * 4;
    return l;
}

}  // namespace dlp
