// fq_attention_window.cu -- paged attention over the last `window` tokens of each sequence and its first `sinks`: the kernels
// of fq_attention.cu, compiled with the window's tiles and masks.
#define FQ_ATTENTION_WINDOW
#include "fq_attention.cu"
