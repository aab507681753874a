// bq_attn.hip -- attention over the 4-bit cache: how a call is cut, and heads of 128 numbers.
#include "bq_attn.h"

namespace bq {

namespace attn {

hipError_t launch_width(std::integral_constant<int, 128>, const Args& a, const AttnPlan& p, bool f16,
                        hipStream_t stream) {
    return launch_any<128>(a, p, f16, stream);
}

}  // namespace attn

AttnPlan attn_plan(int64_t seqs, int64_t rows, int64_t max_q, int64_t max_len, int heads,
                   int kv_heads, int dim, int group) {
    constexpr int kCus = 256;
    AttnPlan p{};
    const int64_t m = max_q * (heads / kv_heads);       // rows of one sequence and cache head
    p.by_rows = m > 64;
    p.cols = !p.by_rows || m <= 128 || dim == 256 ? 1 : 2;
    const int64_t tile = 16 * p.cols * (p.by_rows ? 8 : 1);
    p.tiles = (int)((m + tile - 1) / tile);
    p.splits = 1;
    const int64_t base = seqs * kv_heads * p.tiles;
    if (!p.by_rows) {
        // as many workgroups as the card holds, unless there are units for all of them or too many
        // sequences to add up
        const int64_t most = kCus * attn::tokens_groups(dim, group, true);
        const int64_t turns = base * ((max_len + 127) / 128 + 1);
        if (seqs <= attn::kMaxDealt && base < most && turns < ((int64_t)1 << 31) && max_len > 128) {
            p.dealt = (int)(turns < most ? turns : most);
            p.ws_bytes = p.dealt * (int64_t)(2 * 16 * 4) * (dim + 2) + 4 * (2 * attn::kMaxDealt + 1);
        }
        return p;
    }
    // two workgroups to a compute unit, and 256 tokens or more to a workgroup
    int64_t splits = 2 * kCus / (base > 0 ? base : 1);
    const int64_t longest = (max_len + 255) / 256;
    splits = splits < longest ? splits : longest;
    const int64_t cell = rows * heads * 4 * (dim + 2);
    const int64_t room = ((int64_t)64 << 20) / (cell > 0 ? cell : 1);
    splits = splits < room ? splits : room;
    splits = splits < attn::kMaxSplits ? splits : attn::kMaxSplits;
    p.splits = (int)(splits < 1 ? 1 : splits);
    p.ws_bytes = p.splits > 1 ? p.splits * cell : 0;
    return p;
}

hipError_t launch_attn_i4(const AttnI4& a, const AttnPlan& p, bool f16, hipStream_t stream) {
    attn::Args g{};
    g.a = a;
    using attn::Div;
    g.heads = Div::by(a.c.heads);
    g.by_splits = Div::by(p.splits);
    g.cells = Div::by(a.c.heads * p.splits);
    // new rows that are half of a sequence or less see most of it, each
    g.by_seq = !a.causal || 2 * (int64_t)a.max_q <= a.max_len;
    g.inner = Div::by(g.by_seq ? p.tiles : a.seqs);
    g.groups = (int32_t)((int64_t)a.seqs * p.tiles * a.c.heads * p.splits);
    g.share = Div::by(a.heads / a.c.heads);
    g.bpp = Div::by(a.c.page_size / 8);
    g.tiles = p.tiles;
    g.splits = p.splits;
    g.dealt = p.dealt;
    g.scale2 = a.scale * 1.44269504088896341f;
    if (p.ws_bytes > 0) {
        const int64_t parts = p.dealt ? p.dealt * (int64_t)32 : (int64_t)p.splits * a.rows * a.heads;
        g.part = static_cast<float*>(a.ws);
        g.ml = g.part + parts * a.c.dim;
        g.found = reinterpret_cast<int32_t*>(g.ml + 2 * parts);
    }
    return a.c.dim == 64    ? attn::launch_width(std::integral_constant<int, 64>{}, g, p, f16, stream)
           : a.c.dim == 128 ? attn::launch_width(std::integral_constant<int, 128>{}, g, p, f16, stream)
                            : attn::launch_width(std::integral_constant<int, 256>{}, g, p, f16, stream);
}

}  // namespace bq
