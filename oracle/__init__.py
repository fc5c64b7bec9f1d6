"""Float64 CPU oracle (test infrastructure only; see ``la2_oracle``)."""

from .la2_oracle import (  # noqa: F401
    backward,
    backward_decay,
    backward_gqa,
    backward_rows,
    blocked_forward,
    decode_step,
    backward_from_states,
    forward,
    forward_decay,
    forward_from_state,
    forward_gqa,
    forward_rows,
    kv_state,
    recurrent_forward,
    recurrent_forward_decay,
    relative_frobenius,
)
from .gated_oracle import (  # noqa: E402,F401
    backward_gated,
    forward_gated,
    kv_state_gated,
    qk_norm_rope,
    qk_norm_rope_backward,
    state_compact,
    state_copy,
)
