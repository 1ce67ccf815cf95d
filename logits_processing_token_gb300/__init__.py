"""GB300-native per-step token selection (logits processors, greedy/multinomial
selection, assisted-generation verify) and the attention over a paged cache
that precedes it, as CUDA kernels for sm_103a behind the C ABI of include/tg.h.  This package is the thin Python binding."""
from .tg import (  # noqa: F401
    EXPORTS, TG_DTYPE_BF16, TG_DTYPE_F32, TG_ERR_CUDA, TG_ERR_INVALID_ARGUMENT, TG_ERR_OUT_OF_MEMORY,
    TG_ERR_UNSUPPORTED, TG_FLAG_BAD_ROW, TG_FLAG_BAD_STATE, TG_FLAG_HISTORY_ID_OUT_OF_RANGE, TG_FLAG_SLOW_PATH,
    TG_FLAG_TIMEOUT,
    TG_GREEDY, TG_MAX_PROCESSORS, TG_MAX_STATE_COLS, TG_MAX_VOCAB, TG_NOALLOC_MAX_BATCH, TG_OK, TG_PROC_BIAS,
    TG_PROC_SET, TG_SAMPLE, Config, TGError, load_library, make_params, tg_clear_status, tg_beam_keep, tg_beam_step,
    tg_next_num_candidates, tg_params, tg_process, tg_process_state, tg_query_status, tg_select, tg_select_state,
    tg_set_wait_limit, tg_status_string, tg_status_word, tg_verify, tg_verify_history,
    TG_DTYPE_E4M3, TG_DTYPE_F16, TG_FLAG_BAD_PAGE, TG_MAX_HEAD_DIM, TG_MAX_STEP_TOKENS, TG_PAGES_HEAD_TOKEN,
    TG_PAGES_TOKEN_HEAD, AttnConfig, make_attn_params, tg_attend_prompt, tg_attend_step, tg_attn_clear_status,
    tg_attn_params, tg_attn_status_word, tg_cache, tg_cache_append,
)
