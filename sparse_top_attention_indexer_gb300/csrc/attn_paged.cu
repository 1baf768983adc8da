// attn_paged.cu -- how the attention over a paged cache splits its work, and its kernels for rows of up to 256 dims.
#include "attn_paged.cuh"

namespace sti {

extern template cudaError_t launch_attn_paged_nm<3>(const CUtensorMap&, const AttnPagedParams&, cudaStream_t);   // attn_paged_wide.cu
extern template cudaError_t launch_attn_paged_nm<4>(const CUtensorMap&, const AttnPagedParams&, cudaStream_t);

AttnPagedPlan attn_paged_plan(int B, int s, int h, int d, int cap, int window, int n_first, int num_sms) {
    AttnPagedPlan l;
    l.pack = h <= 32 ? 64 / h : 1;   // as attn_fp4_plan
    if (l.pack > s) l.pack = s;
    l.groups = (s + l.pack - 1) / l.pack;
    int64_t rows = cap;              // of a group's list, at most
    if (window > 0 && (int64_t)window + l.pack - 1 + n_first < rows) rows = (int64_t)window + l.pack - 1 + n_first;
    const int64_t tiles = (rows + kRows - 1) / kRows, groups = (int64_t)B * l.groups;
    // A list of t tiles takes its CTA some 5 us and 1.45 t.  Splitting evens the CTAs' tiles out, but costs as much as another 5 tiles
    // (second kernel; parts written and read), with more queries 13 (several parts per CTA).  Of long lists some may be much longer
    // than others, which only splitting evens out: those are not taken whole.  (All by what the table and the window allow, as the
    // lengths are on the device: 128 queries over 600 rows take 24 us with a table of 1024 positions, 39 with one of 65536.)
    const int64_t waves = (groups + num_sms - 1) / num_sms;
    const double extra = 5.0 + (12 * groups < 8 * num_sms ? 12.0 * groups / num_sms : 8.0);
    l.whole = tiles <= 16 && (double)(waves * tiles) <= (double)(tiles * groups) / num_sms + extra;
    // Pieces of at least two tiles, when the parts of a few queries otherwise take longer to write and join than the tiles
    // (16 queries of 64 heads x 512 over 640 rows 20.7 -> 16.0 us, 8 groups of 4 x 16 heads over 1000 rows 22.8 -> 17.5).
    l.least = groups >= 3 && (l.pack == 1 || d > 128) ? 2 : 1;
    const int64_t list = l.whole ? groups : (tiles * groups + l.least - 1) / l.least;
    l.grid = (int)(list < 1 ? 1 : list < num_sms ? list : num_sms);
    l.by_query = !l.whole && groups <= l.grid;
    return l;
}

cudaError_t launch_attn_paged(const CUtensorMap& tm_q, const AttnPagedParams& p, cudaStream_t stream) {
    switch ((p.d + 127) / 128) {
        case 1: return launch_attn_paged_nm<1>(tm_q, p, stream);
        case 2: return launch_attn_paged_nm<2>(tm_q, p, stream);
        case 3: return launch_attn_paged_nm<3>(tm_q, p, stream);
        default: return launch_attn_paged_nm<4>(tm_q, p, stream);
    }
}

}  // namespace sti
