// Keys that a group of sequences shares, many rows: the kShared form of cross_tiles.cu.
#define PKV_FORM kShared
#define PKV_LAUNCH(suffix) launch_shared##suffix
#include "cross_tiles.cu"
