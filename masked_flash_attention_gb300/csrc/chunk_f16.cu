// chunk_f16.cu -- the fp16 instantiations of the chunk attention kernel (the
// kernel source is shared with chunk_sm103.cu; only the element type differs).
#define MFA_CHUNK_F16_UNIT 1
#include "chunk_sm103.cu"
