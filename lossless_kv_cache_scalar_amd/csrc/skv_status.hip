// skv_status.hip -- the status codes in words.  Contract: skv.h.
#include "skv.h"

extern "C" const char *skv_status_string(int status) {
  switch (status) {
    case SKV_OK: return "ok";
    case SKV_ERR_ARG: return "invalid argument";
    case SKV_ERR_UNSUPPORTED: return "unsupported shape (head_dim must be a multiple of 8 dividing 512)";
    case SKV_ERR_HIP: return "HIP runtime error";
    case SKV_ERR_CAPACITY: return "compressed stream exceeds the output capacity";
    case SKV_ERR_CORRUPT: return "corrupt stream";
    case SKV_ERR_TABLE: return "histogram too large for the p_hat table";
    case SKV_ERR_SCRATCH: return "shape needs more than the library's static scratch (skv_decode_static)";
    case SKV_ERR_PAGES: return "no room in the paged cache (too few free pages, or a table row overflows)";
    default: return "unknown status";
  }
}
