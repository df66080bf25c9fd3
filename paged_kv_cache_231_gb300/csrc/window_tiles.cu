// The same, many rows: the kCausal form of cross_tiles.cu.
#define PKV_FORM kCausal
#define PKV_LAUNCH(suffix) launch_causal##suffix
#include "cross_tiles.cu"
