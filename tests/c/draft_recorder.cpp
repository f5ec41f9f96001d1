// The launches of the drafted step's operators, recorded instead of made: linked with
// draft.cpp, decode.cpp, plan.cpp and decode_recorder.cpp in place of the device code.
#include "draft.h"

namespace detfold_impl {

static int moves;
static CompactArgs compacted;
int launch_tree(const TreeArgs &, void *) { return DETFOLD_OK; }
int launch_copy_pages(const CopyArgs &, int64_t, void *) { return ++moves, DETFOLD_OK; }
int launch_compact(const CompactArgs &a, void *) { return ++moves, compacted = a, DETFOLD_OK; }

}  // namespace detfold_impl

extern "C" int recorded_moves() { return detfold_impl::moves; }
extern "C" int recorded_runs() { return (int)detfold_impl::compacted.runs.d; }     // of the last compaction
extern "C" int recorded_key_runs() { return detfold_impl::compacted.k_runs; }
