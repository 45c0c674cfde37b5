// Status of the decode operators' device words (host).
#include "gs_decode.h"

extern "C" gs_status gs_decode_status_from_word(uint32_t word) {
    if (word & GS_DEV_BAD_SEQ) return GS_ERR_INVALID_ARG;
    if (word & GS_DEV_NO_PAGE) return GS_ERR_CAPACITY;
    if (word & GS_DEV_EMPTY_ROW) return GS_ERR_UNSUPPORTED;
    return gs_status_from_word(word);
}
