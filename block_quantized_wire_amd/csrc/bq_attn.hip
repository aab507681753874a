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
    // Up to 64 rows the waves share the tokens, beyond them the tokens' operands (16 sequences of
    // 4096 tokens, 8 heads of 128 numbers, bf16: 64 rows 44-50 us against 63, 96 rows 69 against 76, 128 rows 88
    // against 80; 2 of 16384, 128 rows: 60 against 48; from 65 to 96 rows the tokens' sharing is up to 10% faster).  Beyond 128 rows a wave has 32 of them (256 rows
    // of 16 x 4096 tokens: 147 us, with 16 rows 176; 128 rows: 110 against 88); at a width of 256
    // their results alone would be half of its registers.
    p.by_rows = m > 64;
    p.cols = !p.by_rows || m <= 128 || dim == 256 ? 1 : 2;
    const int64_t tile = 16 * p.cols * (p.by_rows ? 8 : 1);
    p.tiles = (int)((m + tile - 1) / tile);
    p.splits = 1;
    const int64_t base = seqs * kv_heads * p.tiles;
    if (!p.by_rows) {
        // Turns are dealt out, to as many workgroups as the card holds, where that is worth the join.
        // A unit takes its workgroup some 7 us per 1000 tokens (12 at a width of 256 or with four groups);
        // dealing costs about 10 us, and more the more units there are.  One row, 8 heads of 128 numbers, dealt
        // and not: a sequence of 4096 tokens 14 and 34 us, of 1024 13 and 13, of 512 13 and 10; 16 of
        // 8192 40 and 65, of 2048 23 and 22; 32 of 1000 to 8192 47 and 63, of 8192 67 and 66, of 2048 31
        // and 22; 64 of 4096 68 and 51.
        const int64_t long_by = (384 - base) * max_len * (dim == 256 || dim / group >= 4 ? 2 : 1);
        // The kernels count turns in 32 bits.
        const int64_t turns = base * ((max_len + 127) / 128 + 1);
        if (seqs <= attn::kMaxDealt && base < 384 && long_by > (int64_t)1 << 19 && turns < (int64_t)1 << 31) {
            const int64_t most = kCus * attn::tokens_groups(dim, group, true);
            p.dealt = (int)(turns < most ? turns : most);
            p.ws_bytes = p.dealt * (int64_t)(2 * 16 * 4) * (dim + 2) + 4 * (2 * attn::kMaxDealt + 1);
        }
        return p;
    }
    // As many workgroups as compute units, which have registers for one, and 256 tokens or more to
    // each.  512 rows of 16384 tokens, 8 heads of 128 numbers: 73 us, with twice the workgroups 89; 512
    // of 2048 35, with 128 tokens or more 36, with 512 40.
    int64_t splits = kCus / (base > 0 ? base : 1);
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
    // New rows that are half of a sequence or less see most of it, each (1021 of 1500 to 4096 tokens,
    // four sequences: 228 us by sequence, 310 by tile; of 4096, all four: 345 and 321).
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
