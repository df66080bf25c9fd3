// Causal attention over the paged cache (pkv_paged_window_attention, and the sequences' own keys in
// pkv_paged_prefix_attention), few rows and joins: the kCausal form of cross.cu.
#define PKV_FORM kCausal
#define PKV_LAUNCH(suffix) launch_causal##suffix
#include "cross.cu"
