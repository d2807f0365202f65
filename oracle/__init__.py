"""fp64 CPU oracle (test infrastructure only; never imported by the product path)."""
from .streamkl_oracle import (  # noqa: F401
    allowed,
    oracle_bwd,
    oracle_bwd_gqa,
    oracle_bwd_shard,
    oracle_bwd_teacher,
    oracle_bwd_teacher_gqa,
    oracle_bwd_teacher_shard,
    oracle_bwd_teacher_varlen,
    oracle_bwd_varlen,
    oracle_dk_rows,
    oracle_fwd,
    oracle_fwd_gqa,
    oracle_fwd_varlen,
    oracle_merge_states,
    oracle_partial_state,
    oracle_row_work,
    oracle_rows,
    row_pair_count,
)
from .sparse_oracle import (  # noqa: F401
    oracle_block_mass,
    oracle_block_select,
    oracle_sparse_attn,
    selected_keys,
)
